"""What the operators around a serving step refuse, on the CPU: through the C ABI
with addresses that are never dereferenced, and through the binding with CPU
tensors."""
import struct

import pytest
import torch

import exact_lloyd_means_amd as fk

FAKE, ODD = 0x10000, 0x10001
ROPE, ROWS = struct.Struct("@qiiiiifPP"), struct.Struct("@PPqqqqii")
VERIFY, POOL, CACHE = struct.Struct("@qqqPPPPqqiiPPPPPP"), struct.Struct("@qqqiiPPPPP"), struct.Struct("@PPPqiiii")
ATTN = struct.Struct("@qqiiqqqPPPPfiiPP")
EINVAL, EUNSUPPORTED, EWORKSPACE = fk.FK_EINVAL, fk.FK_EUNSUPPORTED, fk.FK_EWORKSPACE


def rope(T=3, D=128, R=64, dtype=fk.FK_BF16, inter=0, inverse=0, factor=1.0, pos=FAKE, turns=FAKE, n=1, rows=None):
    rows = rows or [{}]
    packed = b"".join(row(**r) for r in rows)
    return fk.lib.fk_rope(ROPE.pack(T, D, R, dtype, inter, inverse, factor, pos or 0, turns or 0), n, packed, None)


def row(x=FAKE, y=FAKE, xt=1024, xh=128, yt=1024, yh=128, heads=8, reserved=0):
    return ROWS.pack(x or 0, y or 0, xt, xh, yt, yh, heads, reserved)


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), EINVAL), (dict(T=(1 << 24) + 1), EUNSUPPORTED), (dict(D=127), EUNSUPPORTED), (dict(D=0), EUNSUPPORTED),
    (dict(D=1026), EUNSUPPORTED), (dict(R=0), EINVAL), (dict(R=63), EINVAL), (dict(R=130), EINVAL), (dict(dtype=3), EUNSUPPORTED),
    (dict(dtype=-1), EUNSUPPORTED), (dict(inter=2), EINVAL), (dict(inverse=-1), EINVAL), (dict(factor=float("nan")), EINVAL),
    (dict(factor=float("inf")), EINVAL), (dict(pos=None), EINVAL), (dict(pos=FAKE + 2), EINVAL), (dict(turns=None), EINVAL),
    (dict(turns=FAKE + 4), EINVAL), (dict(n=0), EINVAL), (dict(n=3), EINVAL), (dict(rows=[dict(x=None)]), EINVAL),
    (dict(rows=[dict(y=None)]), EINVAL), (dict(rows=[dict(x=ODD)]), EINVAL), (dict(dtype=fk.FK_F32, rows=[dict(x=FAKE + 2)]), EINVAL),
    (dict(rows=[dict(heads=0)]), EINVAL), (dict(rows=[dict(heads=65537)]), EUNSUPPORTED), (dict(rows=[dict(xt=-1)]), EINVAL),
    (dict(rows=[dict(yh=-1)]), EINVAL), (dict(rows=[dict(yt=2048)]), EINVAL), (dict(rows=[dict(reserved=1)]), EINVAL),
    (dict(n=2, rows=[{}, dict(heads=-1)]), EINVAL), (dict(rows=[dict(xh=0, yh=0)]), EINVAL), (dict(rows=[dict(yh=127, xh=127)]), EINVAL),
    (dict(rows=[dict(xt=0, yt=0)]), EINVAL), (dict(n=2, rows=[{}, dict(y=FAKE * 2, yh=0)]), EINVAL)])
def test_rope_arguments(kw, status):
    assert rope(**kw) == status
    assert fk.lib.fk_last_error()


def verify(B=2, T=5, V=100, cu=FAKE, tokens=FAKE, p=FAKE, q=FAKE, p_row=100, q_row=100, dtype=fk.FK_F32, reserved=0, u=FAKE, pick=FAKE,
           seq=FAKE, accepted=FAKE, emitted=FAKE, keep=FAKE, ws=FAKE, n=1 << 40):
    args = [x or 0 for x in (cu, tokens, p, q)], [x or 0 for x in (u, pick, seq, accepted, emitted, keep)]
    return fk.lib.fk_verify(VERIFY.pack(B, T, V, *args[0], p_row, q_row, dtype, reserved, *args[1]), ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), EINVAL), (dict(T=0), EINVAL), (dict(V=0), EINVAL), (dict(B=(1 << 20) + 1), EUNSUPPORTED), (dict(T=(1 << 24) + 1), EUNSUPPORTED),
    (dict(V=(1 << 20) + 1), EUNSUPPORTED), (dict(dtype=7), EUNSUPPORTED), (dict(reserved=1), EINVAL), (dict(cu=None), EINVAL),
    (dict(tokens=FAKE + 2), EINVAL), (dict(p=None), EINVAL), (dict(p=FAKE + 2), EINVAL), (dict(q=FAKE + 2), EINVAL), (dict(p_row=-1), EINVAL),
    (dict(q_row=-1), EINVAL), (dict(u=FAKE + 2), EINVAL), (dict(pick=None), EINVAL), (dict(u=None), EINVAL), (dict(u=None, pick=None), EINVAL),
    (dict(accepted=None), EINVAL), (dict(emitted=FAKE + 2), EINVAL), (dict(seq=None), EINVAL), (dict(keep=FAKE + 2), EINVAL),
    (dict(ws=None), EWORKSPACE), (dict(ws=FAKE + 8), EINVAL), (dict(n=8), EWORKSPACE)])
def test_verify_arguments(kw, status):
    assert verify(**kw) == status


def test_verify_workspace():
    size = fk.lib.fk_verify_workspace_bytes
    assert size(0, 1, 1) == size(1, 1, (1 << 20) + 1) == 0
    assert size(1, 1, 1) == 16 + 4
    # a sum for what is left and one for the row, of each piece; a row's largest of each piece
    assert size(64, 384, 128000) >= 64 * 64 * 16 + 64 * 4 and size(1, 1, 1 << 20) <= 4096 * 16 + 4


def pool(R=4, M=8, N=50, P=64, reserved=0, table=FAKE, lens=FAKE, shares=FAKE, free=FAKE, count=FAKE):
    return POOL.pack(R, M, N, P, reserved, *(x or 0 for x in (table, lens, shares, free, count)))


POOLS = [(dict(R=0), EINVAL), (dict(M=0), EINVAL), (dict(N=0), EINVAL), (dict(R=(1 << 20) + 1), EUNSUPPORTED), (dict(P=16), EUNSUPPORTED),
         (dict(P=48), EUNSUPPORTED), (dict(P=2048), EUNSUPPORTED), (dict(M=1 << 26), EUNSUPPORTED), (dict(N=1 << 26), EUNSUPPORTED),
         (dict(reserved=1), EINVAL), (dict(table=None), EINVAL), (dict(lens=FAKE + 2), EINVAL), (dict(shares=None), EINVAL),
         (dict(free=None), EINVAL), (dict(count=FAKE + 1), EINVAL)]


@pytest.mark.parametrize("kw,status", POOLS)
def test_pools(kw, status):
    assert fk.lib.fk_kv_fork(pool(**kw), 2, FAKE, FAKE, FAKE, FAKE, None, FAKE, 1 << 40, None) == status
    assert fk.lib.fk_kv_compact(pool(**kw), FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 20, FAKE, 1 << 40, None) == status


def test_fork_arguments():
    def fork(n=2, rows=FAKE, sources=FAKE, keep=FAKE, copies=FAKE, seq=0, ws=FAKE, size=1 << 40, p=None):
        return fk.lib.fk_kv_fork(p or pool(), n, rows, sources, keep, copies, seq, ws, size, None)
    for kw, status in ((dict(n=0), EINVAL), (dict(n=65537), EUNSUPPORTED), (dict(n=65536, p=pool(M=1 << 16)), EUNSUPPORTED),
                       (dict(rows=None), EINVAL), (dict(rows=ODD), EINVAL), (dict(sources=FAKE + 2), EINVAL), (dict(keep=None), EINVAL),
                       (dict(copies=None), EINVAL), (dict(seq=FAKE + 2), EINVAL), (dict(ws=None), EWORKSPACE), (dict(ws=FAKE + 8), EINVAL),
                       (dict(size=8), EWORKSPACE)):
        assert fork(**kw) == status, kw
    assert fk.lib.fk_kv_fork(None, 2, FAKE, FAKE, FAKE, FAKE, 0, FAKE, 1 << 40, None) == EINVAL
    size = fk.lib.fk_kv_fork_workspace_bytes
    assert size(0, pool()) == 0 and size(3, pool(P=40)) == 0
    assert size(3, pool(table=None)) >= 3 * 8 * 4 + 50 * 20


def test_compact_arguments():
    def compact(table=FAKE, shares=FAKE, free=FAKE, left=FAKE, moves=FAKE, n=25, ws=FAKE, size=1 << 40, p=None):
        return fk.lib.fk_kv_compact(p or pool(), table, shares, free, left, moves, n, ws, size, None)
    for kw, status in ((dict(table=None), EINVAL), (dict(shares=ODD), EINVAL), (dict(free=None), EINVAL), (dict(left=None), EINVAL),
                       (dict(moves=None), EINVAL), (dict(n=24), EINVAL), (dict(n=(1 << 20) + 1), EUNSUPPORTED),
                       (dict(p=pool(N=(1 << 20) + 1)), EUNSUPPORTED), (dict(ws=None), EWORKSPACE), (dict(ws=FAKE + 4), EINVAL),
                       (dict(size=8), EWORKSPACE)):
        assert compact(**kw) == status, kw
    assert fk.lib.fk_kv_compact_workspace_bytes(0) == fk.lib.fk_kv_compact_workspace_bytes((1 << 20) + 1) == 0


def test_copy_arguments():
    c = CACHE.pack(FAKE, FAKE, FAKE, 4, 64, 2, 128, fk.FK_BF16)
    assert fk.lib.fk_kv4_copy(c, 0, FAKE, None) == EINVAL
    assert fk.lib.fk_kv4_copy(c, (1 << 20) + 1, FAKE, None) == EUNSUPPORTED
    assert fk.lib.fk_kv4_copy(c, 1, None, None) == EINVAL
    assert fk.lib.fk_kv4_copy(c, 1, FAKE + 2, None) == EINVAL
    assert fk.lib.fk_kv4_copy(CACHE.pack(FAKE, FAKE, FAKE, 4, 64, 2, 96, fk.FK_BF16), 1, FAKE, None) == EUNSUPPORTED
    assert fk.lib.fk_kv4_copy(CACHE.pack(0, FAKE, FAKE, 4, 64, 2, 128, fk.FK_BF16), 1, FAKE, None) == EINVAL


def test_shared_attention_arguments():
    c = CACHE.pack(FAKE, FAKE, FAKE, 4, 64, 2, 128, fk.FK_BF16)

    def shared(groups=1, cug=FAKE, prefix=FAKE, ws=FAKE, size=1 << 40, **kw):
        a = dict(B=2, T=3, Hq=8, max_q=2, M=4, qt=1024, qh=128, q=FAKE, cu=FAKE, seq=FAKE, table=FAKE, scale=0.1, causal=1, window=0,
                 out=FAKE, lse=0) | kw
        return fk.lib.fk_kv4_attention_shared(c, ATTN.pack(*a.values()), groups, cug, prefix, ws, size, None)
    for kw, status in ((dict(groups=0), EINVAL), (dict(groups=3), EINVAL), (dict(cug=None), EINVAL), (dict(prefix=FAKE + 2), EINVAL),
                       (dict(Hq=7), EINVAL), (dict(max_q=0), EINVAL), (dict(out=0), EINVAL), (dict(scale=0.0), EINVAL),
                       (dict(causal=3), EINVAL), (dict(window=-1), EINVAL), (dict(B=1 << 20, M=1 << 11), EUNSUPPORTED),
                       (dict(ws=None), EWORKSPACE), (dict(ws=FAKE + 8), EINVAL), (dict(size=8), EWORKSPACE)):
        assert shared(**kw) == status, kw
    size = fk.lib.fk_kv4_attn_shared_workspace_bytes
    assert size(c, 4, 4, 8, 1, 0) == size(c, 4, 4, 8, 1, 5) == size(c, 4, 4, 7, 1, 1) == 0
    assert size(c, 4, 4, 8, 1, 1) > 0


# ---- the binding ------------------------------------------------------------------------

def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_binding_of_rope():
    q, pos, turns = torch.zeros(3, 4, 64), i32(3), fk.rope_turns(64, device="cpu")
    for args, kw in (((q[0], None, pos, turns), {}), ((q.double(), None, pos, turns), {}), ((q, q.half(), pos, turns), {}),
                     ((q, torch.zeros(3, 4, 32), pos, turns), {}), ((q, None, pos.long(), turns), {}), ((q, None, i32(4), turns), {}),
                     ((q, None, pos, turns.int()), {}), ((q, None, pos, turns), dict(k_out=q)), ((q, None, pos, turns, q[:2]), {}),
                     ((q.transpose(1, 2), None, pos, turns), {}), ((q, None, pos, turns), {})):
        with pytest.raises(ValueError):
            fk.fk_rope(*args, **kw)                                # the last: not on the GPU
    with pytest.raises(TypeError):
        fk.fk_rope(None, None, pos, turns)
    for kw in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=8, base=0.0), dict(rot_dim=8, stretch=float("inf")),
               dict(rot_dim=8, trained=100, slow=2.0, fast=2.0)):
        with pytest.raises(ValueError):
            fk.rope_turns(device="cpu", **kw)


def test_turns():
    # a turn is 2^64 units: pair 0 advances a radian a position, the others by the powers of the base
    t = fk.rope_turns(8, 16.0, device="cpu")
    want = [2 ** 64 / (2 * 3.141592653589793) / 2 ** i for i in range(4)]
    assert all(abs(a / b - 1) < 2.0 ** -50 for a, b in zip(t.tolist(), want))
    # pair 0 of a base of 1 stretched to more than half a turn: the upper half is negative
    assert fk.rope_turns(2, 1.0, stretch=0.2, device="cpu").tolist()[0] < 0


def test_binding_of_verify():
    p, cu, tokens, b = torch.zeros(4, 10), i32(3), i32(4), i32(2)
    u, pick = torch.zeros(4), torch.zeros(2)
    ok = dict(cu=cu, tokens=tokens, target=p, accepted=b, emitted=tokens)
    for kw in (dict(target=p[0]), dict(target=p.double()), dict(target=p.t()), dict(tokens=tokens.long()), dict(cu=i32(0)), dict(accepted=i32(3)),
               dict(draft=p, accept=u), dict(draft=p.half(), accept=u, pick=pick), dict(draft=p[:3], accept=u, pick=pick),
               dict(accept=u.half(), pick=pick), dict(accept=u, pick=u), dict(keep=b), dict(keep=b, seq_lens=i32(3)), {}):
        with pytest.raises(ValueError):
            fk.fk_verify(**(ok | kw))


def test_binding_of_pages():
    ok = dict(rows=i32(2), sources=i32(2), keep=i32(2), page_size=32, block_table=i32(3, 4), lens=i32(3), shares=i32(9), free_pages=i32(9),
              free_count=i32(1), copies=i32(2, 3))
    for kw in (dict(rows=i32(2).long()), dict(sources=i32(3)), dict(keep=i32(1)), dict(block_table=i32(12)), dict(lens=i32(4)),
               dict(free_pages=i32(8)), dict(free_count=i32(2)), dict(copies=i32(2, 2)), dict(seq=i32(2)), {}):
        with pytest.raises(ValueError):
            fk.fk_kv_fork(**(ok | kw))
    ok = dict(page_size=32, block_table=i32(3, 4), lens=i32(3), shares=i32(9), free_pages=i32(9), free_count=i32(1), new_table=i32(3, 4),
              new_shares=i32(9), new_free=i32(9), free_left=i32(1), moves=i32(5, 3))
    for kw in (dict(new_table=i32(3, 5)), dict(new_shares=i32(8)), dict(new_free=i32(9, 1)), dict(free_left=i32(2)), dict(moves=i32(5, 2)),
               dict(moves=i32(15)), {}):
        with pytest.raises(ValueError):
            fk.fk_kv_compact(**(ok | kw))
    codes, scales = torch.zeros(2, 1, 2, 1, 16 * 64, dtype=torch.uint8), torch.zeros(2, 1, 2, 32).half()
    for args in ((i32(3), codes, scales), (i32(3, 2), codes, scales), (i32(3, 3), codes.int(), scales), (i32(3, 3), codes, scales.float()),
                 (i32(3, 3), codes, scales[:1]), (i32(3, 3), codes, scales)):
        with pytest.raises(ValueError):
            fk.fk_kv4_copy(*args)


def test_binding_of_shared_attention():
    H, D = 2, 64
    ok = dict(q=torch.zeros(3, 4, D).half(), cu_q=i32(3), seq_lens=i32(2), block_table=i32(2, 3), cu_groups=i32(2), prefix_lens=i32(1),
              codebook=torch.zeros(2, H, 16).half(), codes=torch.zeros(5, H, 2, 1, 16 * D, dtype=torch.uint8),
              scales=torch.zeros(5, H, 2, 32).half(), out=torch.zeros(3, 4, D).half(), max_q=2)
    for kw in (dict(cu_groups=i32(1)), dict(prefix_lens=i32(1).long()), dict(cu_groups=i32(2).long()), dict(q=torch.zeros(3, 4, D)),
               dict(block_table=i32(3, 3)), dict(max_q=1 << 40), dict(lse=torch.zeros(3, 4).half()), {}):
        with pytest.raises(ValueError):
            fk.fk_kv4_attention_shared(**(ok | kw))
    with pytest.raises(ValueError):
        fk.kv4_attention_shared_workspace(ok["q"], ok["seq_lens"], i32(3), ok["codes"], 2)
