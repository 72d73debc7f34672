"""What the 4-bit cache refuses, on the CPU: through the C ABI with addresses
that are never dereferenced, and through the binding with CPU tensors."""
import struct

import pytest
import torch

import exact_lloyd_means_amd as fk

FAKE, ODD = 0x10000, 0x10001
CACHE = struct.Struct("@PPPqiiii")
ATTN = struct.Struct("@qqiiqqqPPPPfiiPP")


def cache(codes=FAKE, scales=FAKE, codebook=FAKE, pages=4, page_size=64, heads=2, dim=128, dtype=fk.FK_BF16):
    return CACHE.pack(codes or 0, scales or 0, codebook or 0, pages, page_size, heads, dim, dtype)


def attn(B=2, T=3, Hq=8, max_q=2, max_pages=4, q_token=1024, q_head=128, q=FAKE, cu=FAKE, seq=FAKE, table=FAKE,
         scale=0.1, causal=1, window=0, out=FAKE, lse=0):
    return ATTN.pack(B, T, Hq, max_q, max_pages, q_token, q_head, q or 0, cu or 0, seq or 0, table or 0, scale,
                     causal, window, out or 0, lse)


def call(c=None, a=None, ws=FAKE, ws_bytes=1 << 40):
    return fk.lib.fk_kv4_attention(c or cache(), a or attn(), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(codes=None), fk.FK_EINVAL), (dict(scales=None), fk.FK_EINVAL), (dict(codebook=None), fk.FK_EINVAL),
    (dict(codes=FAKE + 8), fk.FK_EINVAL), (dict(pages=0), fk.FK_EINVAL), (dict(heads=0), fk.FK_EINVAL),
    (dict(page_size=16), fk.FK_EUNSUPPORTED), (dict(page_size=48), fk.FK_EUNSUPPORTED),
    (dict(page_size=2048), fk.FK_EUNSUPPORTED), (dict(dim=96), fk.FK_EUNSUPPORTED),
    (dict(dtype=fk.FK_F32), fk.FK_EUNSUPPORTED), (dict(heads=1025), fk.FK_EUNSUPPORTED),
    (dict(pages=1 << 26), fk.FK_EUNSUPPORTED)])
def test_cache_descriptions(kw, status):
    c = cache(**kw)
    assert call(c=c) == status
    assert fk.lib.fk_kv4_write(c, 1, FAKE, 256, 128, FAKE, 256, 128, FAKE, None) == status
    assert fk.lib.fk_kv4_read(c, 1, FAKE, FAKE, FAKE, None) == status
    assert fk.lib.fk_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), fk.FK_EINVAL), (dict(T=0), fk.FK_EINVAL), (dict(B=(1 << 20) + 1), fk.FK_EUNSUPPORTED),
    (dict(T=(1 << 24) + 1), fk.FK_EUNSUPPORTED), (dict(T=1 << 23), fk.FK_EUNSUPPORTED),
    (dict(Hq=7), fk.FK_EINVAL), (dict(Hq=0), fk.FK_EINVAL), (dict(Hq=2 * 257), fk.FK_EUNSUPPORTED),
    (dict(max_q=0), fk.FK_EINVAL), (dict(max_pages=0), fk.FK_EINVAL), (dict(max_pages=1 << 26), fk.FK_EUNSUPPORTED),
    (dict(B=1 << 20, max_pages=1 << 11), fk.FK_EUNSUPPORTED),
    (dict(q=None), fk.FK_EINVAL), (dict(q=ODD), fk.FK_EINVAL), (dict(cu=None), fk.FK_EINVAL),
    (dict(seq=FAKE + 2), fk.FK_EINVAL), (dict(table=None), fk.FK_EINVAL), (dict(out=None), fk.FK_EINVAL),
    (dict(out=FAKE + 8), fk.FK_EINVAL), (dict(lse=FAKE + 2), fk.FK_EINVAL), (dict(q_token=-1), fk.FK_EINVAL),
    (dict(scale=0.0), fk.FK_EINVAL), (dict(scale=float("nan")), fk.FK_EINVAL), (dict(scale=float("inf")), fk.FK_EINVAL),
    (dict(scale=-1.0), fk.FK_EINVAL), (dict(causal=2), fk.FK_EINVAL), (dict(window=-1), fk.FK_EINVAL)])
def test_attention_arguments(kw, status):
    assert call(a=attn(**kw)) == status


def test_attention_workspace():
    assert call(ws=None) == fk.FK_EWORKSPACE
    assert call(ws=FAKE + 8) == fk.FK_EINVAL
    assert call(ws_bytes=8) == fk.FK_EWORKSPACE
    assert b"needs" in fk.lib.fk_last_error()
    n = fk.lib.fk_kv4_attn_workspace_bytes(cache(codes=0), 64, 64, 8, 1)
    assert n > 0
    # one size serves a call with any block table
    assert call(a=attn(B=64, T=64, max_q=1, max_pages=1 << 14), ws_bytes=n - 1) == fk.FK_EWORKSPACE
    assert fk.lib.fk_kv4_attn_workspace_bytes(cache(dim=80), 64, 64, 8, 1) == 0
    assert fk.lib.fk_kv4_attn_workspace_bytes(cache(), 0, 64, 8, 1) == 0
    assert fk.lib.fk_kv4_attention(None, attn(), FAKE, 1 << 40, None) == fk.FK_EINVAL
    assert fk.lib.fk_kv4_attention(cache(), None, FAKE, 1 << 40, None) == fk.FK_EINVAL


def test_row_arguments():
    w, r, c = fk.lib.fk_kv4_write, fk.lib.fk_kv4_read, cache()
    assert w(c, 0, FAKE, 256, 128, FAKE, 256, 128, FAKE, None) == fk.FK_EINVAL
    assert w(c, 1 << 25, FAKE, 256, 128, FAKE, 256, 128, FAKE, None) == fk.FK_EUNSUPPORTED
    assert w(cache(heads=1024), 1 << 18, FAKE, 256, 128, FAKE, 256, 128, FAKE, None) == fk.FK_EUNSUPPORTED
    assert w(c, 1, None, 256, 128, FAKE, 256, 128, FAKE, None) == fk.FK_EINVAL
    assert w(c, 1, FAKE, 256, 128, ODD, 256, 128, FAKE, None) == fk.FK_EINVAL
    assert w(c, 1, FAKE, 256, -128, FAKE, 256, 128, FAKE, None) == fk.FK_EINVAL
    assert w(c, 1, FAKE, 256, 128, FAKE, -256, 128, FAKE, None) == fk.FK_EINVAL
    assert w(c, 1, FAKE, 256, 128, FAKE, 256, 128, None, None) == fk.FK_EINVAL
    assert r(c, 1, FAKE, FAKE + 8, FAKE, None) == fk.FK_EINVAL
    assert r(c, 1, FAKE, FAKE, None, None) == fk.FK_EINVAL
    assert r(c, 1, FAKE + 2, FAKE, FAKE, None) == fk.FK_EINVAL


PLAN = dict(B=2, max_pages=4, page_size=64, ctx=FAKE, new=FAKE, free=FAKE, free_cap=3, count=FAKE, table=FAKE,
            seq=FAKE, cu=FAKE, slots=FAKE, pos=FAKE, slot_cap=5, left=FAKE, status=FAKE, ws=FAKE, ws_bytes=1 << 20)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), fk.FK_EINVAL), (dict(B=(1 << 20) + 1), fk.FK_EUNSUPPORTED), (dict(page_size=31), fk.FK_EUNSUPPORTED),
    (dict(max_pages=0), fk.FK_EINVAL), (dict(free_cap=-1), fk.FK_EINVAL), (dict(slot_cap=-1), fk.FK_EINVAL),
    (dict(slot_cap=1 << 31), fk.FK_EUNSUPPORTED), (dict(pos=FAKE + 2), fk.FK_EINVAL),
    (dict(ws_bytes=8), fk.FK_EWORKSPACE), (dict(ws=None), fk.FK_EWORKSPACE), (dict(ws=FAKE + 4), fk.FK_EINVAL),
    *[({k: None}, fk.FK_EINVAL) for k in ("ctx", "new", "free", "count", "table", "seq", "cu", "slots", "left", "status")]])
def test_plan_arguments(kw, status):
    assert fk.lib.fk_kv_plan(*{**PLAN, **kw}.values(), None) == status
    assert fk.lib.fk_kv_plan_workspace_bytes(0) == 0


# ---- binding ---------------------------------------------------------------------

H, D, P, T, B = 2, 64, 32, 5, 3


def good(dtype=torch.float16):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    return dict(codes=torch.zeros(4, H, 2, P // 32, 16 * D, dtype=torch.uint8), scales=torch.zeros(4, H, 2, P, dtype=dtype),
                codebook=torch.zeros(2, H, 16, dtype=torch.float16), k=torch.zeros(T, H, D, dtype=dtype),
                v=torch.zeros(T, H, D, dtype=dtype), q=torch.zeros(T, 4 * H, D, dtype=dtype),
                out=torch.zeros(T, 4 * H, D, dtype=dtype), slots=i(T), cu=i(B + 1), seq=i(B), table=i(B, 2),
                lse=torch.zeros(T, 4 * H))


def write(t):
    fk.fk_kv4_write(t["k"], t["v"], t["slots"], t["codebook"], t["codes"], t["scales"])


def read(t):
    fk.fk_kv4_read(t["slots"], t["codebook"], t["codes"], t["scales"], t["k"], t["v"])


def attend(t):
    fk.fk_kv4_attention(t["q"], t["cu"], t["seq"], t["table"], t["codebook"], t["codes"], t["scales"], t["out"], 2,
                        lse=t["lse"])


@pytest.mark.parametrize("f", [write, read, attend])
def test_correct_cpu_tensors_are_rejected_only_for_their_device(f):
    with pytest.raises(ValueError, match="on the GPU"):
        f(good())


@pytest.mark.parametrize("f,which,bad,match", [
    (write, "codes", torch.zeros(4, H, 2, 1, 16 * D), "codes must be uint8"),
    (write, "codes", torch.zeros(4, H, 2, 16 * D, dtype=torch.uint8), "codes must have 5 dimensions"),
    (write, "codes", torch.zeros(4, H, 2, 1, 32 * D, dtype=torch.uint8)[..., ::2], "contiguous"),
    (write, "scales", torch.zeros(4, H, 2, P), "scales must be torch.float16 or"),
    (write, "scales", torch.zeros(4, H, 2, 2 * P, dtype=torch.float16), "scales must have shape"),
    (write, "codebook", torch.zeros(2, H, 16), "codebook must be torch.float16"),
    (write, "codebook", torch.zeros(2, H, 15, dtype=torch.float16), "codebook must have shape"),
    (write, "k", torch.zeros(T, H, D, dtype=torch.bfloat16), "k must be torch.float16"),
    (write, "v", torch.zeros(T, H, D + 1, dtype=torch.float16), "v must have shape"),
    (write, "v", torch.zeros(T, D, H, dtype=torch.float16).transpose(1, 2), "last dimension of v"),
    (write, "slots", torch.zeros(T, dtype=torch.int64), "slots must be torch.int32"),
    (read, "k", torch.zeros(T, H, 2 * D, dtype=torch.float16)[..., :D], "k must be contiguous"),
    (read, "v", torch.zeros(T + 1, H, D, dtype=torch.float16), "v must have shape"),
    (attend, "q", torch.zeros(T, 4 * H, 2 * D, dtype=torch.float16), "q must have shape"),
    (attend, "q", torch.zeros(T, 4 * H, D), "q must be torch.float16"),
    (attend, "out", torch.zeros(T, 4 * H, D, dtype=torch.bfloat16), "out must be torch.float16"),
    (attend, "cu", torch.zeros(B, dtype=torch.int32), "cu_q must have shape"),
    (attend, "table", torch.zeros(B + 1, 2, dtype=torch.int32), "block_table must have shape"),
    (attend, "lse", torch.zeros(T, 4 * H, dtype=torch.float64), "lse must be torch.float32"),
])
def test_binding_rejects(f, which, bad, match):
    t = good()
    t[which] = bad
    with pytest.raises(ValueError, match=match):
        f(t)


def test_binding_rejects_what_is_no_tensor():
    for which in ("codes", "scales", "codebook", "k", "slots"):
        with pytest.raises((TypeError, ValueError)):
            write({**good(), which: None})
    with pytest.raises(TypeError, match="k must be a torch tensor"):
        write({**good(), "k": [1, 2]})


def test_plan_binding():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    args = [i(B), i(B), 32, i(9), i(1), i(B, 4), i(B), i(B + 1), i(7), i(7), i(1), i(4)]
    with pytest.raises(ValueError, match="on the GPU"):
        fk.fk_kv_plan(*args)
    for at, bad, match in ((1, i(B + 1), "new_lens must have shape"), (4, i(2), "free_count must have shape"),
                           (5, i(B), "block_table must have 2 dimensions"), (7, i(B), "cu_new must have shape"),
                           (9, i(6), "positions must have shape"), (11, i(3), "status must have shape"),
                           (0, i(B).long(), "ctx_lens must be torch.int32")):
        with pytest.raises(ValueError, match=match):
            fk.fk_kv_plan(*[bad if j == at else a for j, a in enumerate(args)])


def test_workspaces_of_wrong_sizes():
    t = good()
    with pytest.raises(ValueError, match="head_dim"):
        fk.kv4_attention_workspace(torch.zeros(T, 8, 48, dtype=torch.float16), t["seq"], t["codes"], 1)


def test_cache_class_refuses():
    cb = good()["codebook"]
    with pytest.raises(ValueError, match="page_size"):
        fk.KV4Cache(4, 40, H, D, cb, 2, 100, device="cpu")
    with pytest.raises(ValueError, match="dtype"):
        fk.KV4Cache(4, 32, H, D, cb, 2, 100, dtype=torch.float32, device="cpu")
