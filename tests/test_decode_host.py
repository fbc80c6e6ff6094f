"""Refusals of the decode-step entry points: every bad argument is answered
with its status before anything is enqueued.  No GPU: the pointers below are
never dereferenced, and the binding's checks run on CPU tensors."""
import pytest

A = 0x10000  # a 256-byte-aligned fake address


@pytest.fixture(scope="module")
def L():
    from deterministic_w8a8_int8_gb300 import build
    build.build()
    import deterministic_w8a8_int8_gb300 as p
    return p.lib()


CACHE = dict(k_codes=A, v_codes=A, k_scale=A, v_scale=A)
TABLE = dict(table=A, ld_table=8, lens=A)
GEOM = dict(num_pages=9, max_pages=8, H=2, D=128, block=64)


def append(L, **kw):
    d = dict(k=A, ldk_t=256, ldk_h=128, v=A, ldv_t=256, ldv_h=128, k_open=A, v_open=A, cu=None, S=3, T=3, max_new=1,
             err=None, **CACHE, **TABLE, **GEOM)
    d.update(kw)
    return L.prism_kv_append(d["k"], d["ldk_t"], d["ldk_h"], d["v"], d["ldv_t"], d["ldv_h"], d["k_codes"],
                             d["v_codes"], d["k_scale"], d["v_scale"], d["k_open"], d["v_open"], d["table"],
                             d["ld_table"], d["lens"], d["cu"], d["S"], d["T"], d["max_new"], d["num_pages"],
                             d["max_pages"], d["H"], d["D"], d["block"], d["err"], None)


def attention(L, **kw):
    d = dict(q=A, ldq_t=512, ldq_h=128, out=A, ldo_t=512, ldo_h=128, lse=None, cu=None, scale=0.1, causal=1, window=0,
             S=3, T=3, max_q=1, Hq=4, ws=A, ws_bytes=1 << 40, err=None, **CACHE, **TABLE, **GEOM)
    d.update(kw)
    return L.prism_kv_attention(d["q"], d["ldq_t"], d["ldq_h"], d["k_codes"], d["v_codes"], d["k_scale"],
                                d["v_scale"], d["table"], d["ld_table"], d["lens"], d["cu"], d["out"], d["ldo_t"],
                                d["ldo_h"], d["lse"], d["scale"], d["causal"], d["window"], d["S"], d["T"],
                                d["max_q"], d["num_pages"], d["max_pages"], d["Hq"], d["H"], d["D"], d["block"],
                                d["ws"], d["ws_bytes"], d["err"], None)


BAD_CACHE = [(dict(k_codes=None), -1), (dict(v_codes=None), -1), (dict(k_scale=None), -1), (dict(v_scale=None), -1),
             (dict(table=None), -1), (dict(lens=None), -1), (dict(ld_table=7), -1), (dict(num_pages=0), -1),
             (dict(max_pages=0), -1), (dict(H=0), -1), (dict(block=0), -3), (dict(block=48), -3), (dict(block=8), -3),
             (dict(block=256), -3), (dict(D=96), -3), (dict(D=0), -3), (dict(S=-1), -1), (dict(T=-1), -1),
             (dict(T=4), -1), (dict(k_codes=A + 8), -2), (dict(v_codes=A + 4), -2), (dict(k_scale=A + 2), -2),
             (dict(table=A + 2), -2), (dict(lens=A + 1), -2), (dict(cu=A + 2), -2), (dict(err=A + 2), -2),
             (dict(num_pages=1 << 31), -3), (dict(max_pages=1 << 26, ld_table=1 << 26), -3)]


@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(k=None), -1), (dict(v=None), -1), (dict(k_open=None), -1), (dict(v_open=None), -1), (dict(max_new=0), -1),
    (dict(ldk_t=120), -1), (dict(ldv_h=120), -1), (dict(ldk_t=260), -2), (dict(ldv_h=132), -2), (dict(k=A + 8), -2),
    (dict(v=A + 2), -2), (dict(k_open=A + 8), -2), (dict(v_open=A + 4), -2)])
def test_append_refusals(L, kw, status):
    assert append(L, **kw) == status


@pytest.mark.parametrize("kw,status", BAD_CACHE + [
    (dict(q=None), -1), (dict(out=None), -1), (dict(max_q=0), -1), (dict(ldq_t=120), -1), (dict(ldo_h=120), -1),
    (dict(ldq_t=516), -2), (dict(ldo_h=132), -2), (dict(q=A + 8), -2), (dict(out=A + 2), -2), (dict(lse=A + 2), -2),
    (dict(Hq=3), -1), (dict(Hq=0), -1), (dict(window=-1), -1), (dict(window=4, causal=0), -1), (dict(causal=2), -1),
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1)])
def test_attention_refusals(L, kw, status):
    assert attention(L, **kw) == status


def test_attention_workspace(L):
    need = lambda S, T, max_q, max_pages, Hq=4, H=2, D=128, block=64: L.prism_kv_attention_workspace_bytes(  # noqa: E731
        S, T, max_q, max_pages, Hq, H, D, block)
    assert need(0, 0, 1, 8) == 0 and need(3, 3, 1, 0) == 0 and need(3, 3, 1, 8, Hq=3) == 0 and need(3, 3, 1, 8, D=96) == 0
    big = need(3, 3, 1, 2048)
    if big:
        assert attention(L, max_pages=2048, ld_table=2048, ws=None, ws_bytes=0) == -4
        assert attention(L, max_pages=2048, ld_table=2048, ws_bytes=big - 1) == -4
        assert attention(L, max_pages=2048, ld_table=2048, ws=A + 16) == -2


def test_empty_calls_enqueue_nothing(L):
    assert append(L, S=0, T=0) == 0 and append(L, T=0, cu=A) == 0
    assert attention(L, S=0, T=0) == 0 and attention(L, T=0, cu=A) == 0
    assert w4g(L, M=0) == 0 and w4g(L, N=0) == 0
    assert logprobs(L, R=0) == 0


def w4g(L, **kw):
    d = dict(q=A, ldq=256, a=A, w4=A, ldw4=128, s=A, lds=8, b=None, ldb=0, res=None, ldr=0, out=A, ldo=64, M=2, N=64,
             K=256, g=32)
    d.update(kw)
    return L.prism_w4g_linear(d["q"], d["ldq"], d["a"], d["w4"], d["ldw4"], d["s"], d["lds"], d["b"], d["ldb"],
                              d["res"], d["ldr"], d["out"], d["ldo"], d["M"], d["N"], d["K"], d["g"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), -1), (dict(a=None), -1), (dict(w4=None), -1), (dict(s=None), -1), (dict(out=None), -1),
    (dict(M=-1), -1), (dict(N=-1), -1), (dict(K=0), -1), (dict(g=0), -1), (dict(g=16), -3), (dict(g=256), -3),
    (dict(K=272, ldq=272, ldw4=144), -1), (dict(ldq=240), -1), (dict(ldw4=112), -1), (dict(lds=7), -1),
    (dict(ldo=63), -1), (dict(b=A, ldb=7), -1), (dict(res=A, ldr=63), -1), (dict(ldq=264), -2), (dict(ldw4=136), -2),
    (dict(q=A + 8), -2), (dict(w4=A + 8), -2), (dict(a=A + 2), -2), (dict(s=A + 1), -2), (dict(b=A + 1, ldb=8), -2),
    (dict(res=A + 1, ldr=64), -2), (dict(out=A + 1), -2),
    (dict(K=133248, ldq=133248, ldw4=66624, lds=4164), -3)])
def test_w4g_refusals(L, kw, status):
    assert w4g(L, **kw) == status


def logprobs(L, **kw):
    d = dict(x=A, f32=0, ldl=1000, ids=A, ld_ids=1, n=1, R=2, V=1000, k=5, lp=A, ent=A, ti=A, tl=A, err=None)
    d.update(kw)
    return L.prism_token_logprobs(d["x"], d["f32"], d["ldl"], d["ids"], d["ld_ids"], d["n"], d["R"], d["V"], d["k"],
                                  d["lp"], d["ent"], d["ti"], d["tl"], d["err"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(ids=None), -1), (dict(lp=None), -1), (dict(ti=None), -1), (dict(tl=None), -1),
    (dict(R=-1), -1), (dict(V=0), -1), (dict(n=-1), -1), (dict(k=-1), -1), (dict(V=4, k=5, ldl=4), -1),
    (dict(ldl=999), -1), (dict(ld_ids=0), -1), (dict(f32=2), -1), (dict(k=33), -3), (dict(R=1 << 28), -3),
    (dict(V=1 << 31, ldl=1 << 31), -3), (dict(x=A + 1), -2), (dict(x=A + 2, f32=1), -2), (dict(ids=A + 2), -2),
    (dict(lp=A + 1), -2), (dict(ent=A + 1), -2), (dict(ti=A + 2), -2), (dict(tl=A + 2), -2), (dict(err=A + 1), -2)])
def test_logprobs_refusals(L, kw, status):
    assert logprobs(L, **kw) == status


def test_binding_refuses_cpu_tensors_and_others():
    import torch
    import deterministic_w8a8_int8_gb300 as p
    cache = p.new_kv_cache(4, 2, 64, 16, 1, device="cpu")
    row = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: p.prism_kv_append(row, row, cache, table, lens),
                 lambda: p.prism_kv_attention(row, cache, table, lens),
                 lambda: p.prism_w4g_linear(torch.zeros((1, 32), dtype=torch.int8), torch.zeros(1),
                                            torch.zeros((4, 16), dtype=torch.uint8),
                                            torch.zeros((4, 1), dtype=torch.float16)),
                 lambda: p.prism_token_logprobs(torch.zeros((1, 8)), torch.zeros((1, 1), dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with pytest.raises(TypeError):
        p.prism_kv_append(None, row, cache, table, lens)
    with pytest.raises(AttributeError):
        p.prism_no_such_entry
