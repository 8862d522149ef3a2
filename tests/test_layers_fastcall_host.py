"""The fast-call module's entries of the operators around a layer's products give
the statuses that ctypes gives, and refuse what they cannot convert."""

import pytest

import strided_gemm_gb300 as sg
from tests.test_layers_host import A, B, C, D, E, F, built, fp8, quantise, rope, rope_back, shared  # noqa: F401

CASES = [(fp8, dict(type_c=0)), (fp8, dict(M=0)), (fp8, dict(C=A)), (fp8, dict(a=dict(group=64))), (fp8, dict(rsC=63)),
         (quantise, dict(X=0)), (quantise, dict(K=0)), (quantise, dict(y=dict(data=C))), (rope, dict(dims=63)),
         (rope, dict(part=dict(x=0))), (rope, dict(second=dict(x=F))), (rope, dict(tokens=0)), (rope, dict(interleaved=2)),
         (rope_back, dict(type=0)), (rope_back, dict(part=dict(dx=D))), (rope_back, dict(tokens=0)),
         (rope_back, dict(workspace=F + 8, workspace_bytes=1 << 20)), (shared, dict(N=129)), (shared, dict(O=F)),
         (shared, dict(n_seqs=0)), (shared, dict(n_groups=1 << 30))]


def need_fast():
    if sg._fast is None:
        pytest.skip("the fast-call module is not built (no Python headers)")


def test_statuses_match_ctypes(monkeypatch):
    need_fast()
    fast = [f(**kw) for f, kw in CASES]
    monkeypatch.setattr(sg, "_fast", None)
    assert fast == [f(**kw) for f, kw in CASES]


def test_what_cannot_be_converted_is_refused():
    need_fast()
    f = sg._fast
    part = (A, 1024, 64, B, 1024, 64, 16, 64, 64, 0, C)
    rest = (D, 8, E, 64, 1.0, 0, 1e-6, 0)
    back = (A, 1, 1, B, 1, 1, C, 1, 1, 16, 64, 64, 0, D, 0)
    more = (D, 8, E, 64, 1.0, 0, 1e-6, 0, 0, 0)
    for call in (lambda: f.fp8(1), lambda: f.quantize(1), lambda: f.rope(1), lambda: f.rope_back(1), lambda: f.shared(1),
                 lambda: f.bind_layers(1), lambda: f.rope(2, [part], *rest), lambda: f.rope(2, (part,) * 5, *rest),
                 lambda: f.rope(2, (list(part),), *rest), lambda: f.rope(2, (part[:-1],), *rest),
                 lambda: f.rope("2", (part,), *rest), lambda: f.rope(2, (part,), "D", *rest[1:]),
                 lambda: f.rope(2, (part,), *rest[:4], "1", *rest[5:]), lambda: f.rope_back(2, (back[:-1],), *more),
                 lambda: f.rope_back(2, (back,) * 5, *more), lambda: f.rope_back(2, (back,), *more[:-1])):
        with pytest.raises(TypeError):
            call()
