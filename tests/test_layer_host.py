"""Refusals of the operators between a layer's linears: every bad argument is
answered with its status before anything is enqueued.  No GPU: the pointers
below are never dereferenced, and the binding's checks run on CPU tensors."""
import pytest

A = 0x10000  # a 256-byte-aligned fake address


@pytest.fixture(scope="module")
def L():
    from deterministic_w8a8_int8_gb300 import build
    build.build()
    import deterministic_w8a8_int8_gb300 as p
    return p.lib()


def norm(L, **kw):
    d = dict(x=A, ldx=256, delta=2 * A, ldd=256, alpha=1.0, post=None, w=A, eps=1e-6, M=3, K=256, h=A, ldh=256, form=0, q=A, ldq=256, s=A)
    d.update(kw)
    return L.prism_norm_quant(d["x"], d["ldx"], d["delta"], d["ldd"], d["alpha"], d["post"], d["w"], d["eps"], d["M"], d["K"],
                              d["h"], d["ldh"], d["form"], d["q"], d["ldq"], d["s"], None)


def head(L, **kw):
    d = dict(x=A, ldx=256, w=A, gate=A, ldg=256, inv=None, eps=1e-6, M=3, H=4, D=64, form=0, q=A, ldq=256, s=A)
    d.update(kw)
    return L.prism_head_norm_quant(d["x"], d["ldx"], d["w"], d["gate"], d["ldg"], d["inv"], d["eps"], d["M"], d["H"], d["D"],
                                   d["form"], d["q"], d["ldq"], d["s"], None)


def glu(L, **kw):
    d = dict(x=A, ldx=512, inv=None, M=3, F=256, form=0, q=A, ldq=256, s=A)
    d.update(kw)
    return L.prism_glu_quant(d["x"], d["ldx"], d["inv"], d["M"], d["F"], d["form"], d["q"], d["ldq"], d["s"], None)


def linear(L, **kw):
    d = dict(q=A, ldq_t=256, ldq_h=128, k=A, ldk_t=256, ldk_h=128, v=A, ldv_t=512, ldv_h=128, g=A, ldd=4, state=A, si=A, so=A,
             cu=A, out=A, ldo_t=512, ldo_h=128, scale=0.1, S=3, T=2000, max_len=2000, slots=5, hk=2, hv=4, dk=128, dv=128, ws=A,
             bytes=1 << 40, err=None)
    d.update(kw)
    return L.prism_linear_attention(d["q"], d["ldq_t"], d["ldq_h"], d["k"], d["ldk_t"], d["ldk_h"], d["v"], d["ldv_t"],
                                    d["ldv_h"], d["g"], d["ldd"], d["state"], d["si"], d["so"], d["cu"], d["out"], d["ldo_t"],
                                    d["ldo_h"], d["scale"], d["S"], d["T"], d["max_len"], d["slots"], d["hk"], d["hv"], d["dk"],
                                    d["dv"], d["ws"], d["bytes"], d["err"], None)


CODES = [(dict(q=None), -1), (dict(s=None), -1), (dict(form=2), -1), (dict(form=3, s=None), -1), (dict(form=-1), -1),
         (dict(ldq=240), -1), (dict(ldq=264), -2), (dict(form=1, ldq=260), -2), (dict(q=A + 8), -2), (dict(s=A + 2), -2),
         (dict(M=-1), -1), (dict(x=None), -1), (dict(x=A + 8), -2)]


@pytest.mark.parametrize("kw,status", CODES + [
    (dict(K=0), -1), (dict(K=250, ldx=256), -3), (dict(K=8), -3), (dict(K=32784, ldx=32784, ldd=32784, ldh=32784, ldq=32784), -3),
    (dict(ldx=248), -1), (dict(ldx=260), -2), (dict(w=None), -1), (dict(w=A + 4), -2), (dict(eps=0.0), -1), (dict(eps=2.0), -1),
    (dict(eps=float("nan")), -1), (dict(alpha=float("nan")), -1), (dict(alpha=float("inf")), -1), (dict(h=None), -1),
    (dict(delta=None), -1), (dict(delta=None, h=None, post=A), -1), (dict(post=A + 8), -2), (dict(ldd=200), -1),
    (dict(ldh=200), -1), (dict(ldh=264), -1), (dict(h=2 * A, ldh=264), -1), (dict(delta=A + 2), -2), (dict(h=A + 8), -2), (dict(ldh=260), -2)])
def test_norm_refusals(L, kw, status):
    assert norm(L, **kw) == status


@pytest.mark.parametrize("kw,status", CODES + [
    (dict(D=96), -3), (dict(D=32), -3), (dict(D=0), -1), (dict(H=0), -1), (dict(H=1024, ldq=65536), -3), (dict(H=1 << 40), -3),
    (dict(ldx=248), -1), (dict(ldx=260), -2), (dict(ldg=248), -1), (dict(ldg=260), -2), (dict(gate=A + 8), -2),
    (dict(w=None), -1), (dict(w=A + 8), -2), (dict(inv=A + 4), -2), (dict(eps=0.0), -1)])
def test_head_norm_refusals(L, kw, status):
    assert head(L, **kw) == status


@pytest.mark.parametrize("kw,status", CODES + [
    (dict(F=0), -1), (dict(F=248), -3), (dict(F=32784, ldx=65568, ldq=32784), -3), (dict(ldx=504), -1), (dict(ldx=516), -2),
    (dict(inv=A + 8), -2)])
def test_glu_refusals(L, kw, status):
    assert glu(L, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(S=-1), -1), (dict(T=-1), -1), (dict(max_len=0), -1), (dict(slots=-1), -1), (dict(cu=None), -1), (dict(hk=0), -1),
    (dict(hv=0), -1), (dict(hk=3), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(dk=96), -3),
    (dict(dv=256), -3), (dict(S=1 << 25), -3), (dict(S=1 << 24, hv=32, ldd=32), -3), (dict(T=1 << 31), -3), (dict(hv=1 << 16, ldd=1 << 16), -3),
    (dict(slots=1 << 31), -3), (dict(state=None), -1), (dict(slots=0), -1), (dict(state=None, si=None), -1), (dict(q=None), -1),
    (dict(k=None), -1), (dict(v=None), -1), (dict(out=None), -1), (dict(g=None), -1), (dict(ldd=3), -1), (dict(ldd=-1), -1),
    (dict(ldq_t=64), -1), (dict(ldk_h=120), -1), (dict(ldv_t=516), -2), (dict(ldo_h=132), -2), (dict(q=A + 8), -2),
    (dict(out=A + 2), -2), (dict(g=A + 2), -2), (dict(state=A + 8), -2), (dict(si=A + 2), -2), (dict(so=A + 1), -2),
    (dict(cu=A + 2), -2), (dict(err=A + 2), -2), (dict(ws=None), -4), (dict(bytes=1 << 10), -4), (dict(ws=A + 16), -2)])
def test_linear_refusals(L, kw, status):
    assert linear(L, **kw) == status


def test_nothing_to_do(L):
    assert norm(L, M=0, x=None) == 0 and head(L, M=0) == 0 and glu(L, M=0) == 0 and linear(L, S=0) == 0


def test_workspace(L):
    """None for calls that are not cut into segments; else a place of states for each 512 tokens at most."""
    f = L.prism_linear_attention_workspace_bytes
    assert f(64, 64, 1, 40, 128, 128) == 0 and f(1, 1535, 1535, 40, 128, 128) == 0 and f(0, 0, 1, 40, 128, 128) == 0
    assert f(1, 1536, 1536, 40, 128, 96) == 0
    one = 40 * (128 * 128 + 4) * 4
    assert f(1, 1536, 1536, 40, 128, 128) == 3 * one
    assert f(3, 8191, 8191, 40, 128, 128) <= 16 * one
    assert f(1, 1 << 20, 1 << 20, 400, 128, 128) == 0     # heads enough
    assert f(1, 767, 767, 8, 128, 128) == 0 and f(1, 768, 768, 8, 128, 128) == 3 * 8 * (128 * 128 + 4) * 4
    assert f(1, 767, 767, 8, 64, 64) == 0 and f(1, 768, 768, 8, 64, 64) == 3 * 8 * (64 * 64 + 4) * 4


@pytest.mark.parametrize("call,text", [
    (lambda p, t: p.prism_norm_quant(t.zeros(2, 64), t.zeros(64)), "CUDA device"),
    (lambda p, t: p.prism_norm_quant([1], t.zeros(64)), "torch.Tensor"),
    (lambda p, t: p.prism_head_norm_quant(t.zeros(2, 1, 64), t.zeros(64, 1)), "1 dims"),
    (lambda p, t: p.prism_glu_quant(t.zeros(2, 64)), "CUDA device"),
    (lambda p, t: p.prism_linear_attention(t.zeros(2, 1, 64), t.zeros(2, 1, 64), t.zeros(2, 1, 64), t.zeros(1)), "CUDA device"),
])
def test_binding_refusals(L, call, text):
    import torch

    import deterministic_w8a8_int8_gb300 as p
    with pytest.raises((TypeError, ValueError), match=text):
        call(p, torch)
