"""The 8-bit K/V cache on the GPU (vla_kv8_* through the binding) against the fp64 model.

Stored values are compared bit for bit (a rounding to nearest of an exact quotient). The
attention's bound, element by element: the output's own rounding to bf16, half a step =
2^-8 |o|; the weights' rounding, at most 2^-8 of each (the coarser of the two kernels: bf16
with many query rows, half a step 2^-8; fp16 with few, 2^-11), and the scores' error e_s, both
of which reach o through sum p |v| / sum p:
    |err| <= 2^-8 |o| + (2^-8 + 2 e_s) * mean|v| (1 + 2^-7)
                 + 448 * 2^-22 * top + 2^-133
with e_s = scale * ((D + 8) * 2^-23 * max_j sum_d |q_d k_jd| + 2^-17 max|q| max_j sum_d |k_jd|)
+ 2^-20 (fp32 sums of exact products, truncated at worst; Q as two E4M3 terms of a row scaled
to a largest value in [128, 256), off by at most half of E4M3's smallest step, 2^-10; exp2
and the subtraction of the reference, 2^-20 in all). The last terms are the ends of the number
ranges: fp16 weights are held relative to the largest of their block, with a smallest step of
2^-24 (bf16's range has no such end here), so each of n keys adds less than 2^-22 of the
largest weight times its V scale times 448 (top = n * largest weight * V scale); bf16 ends at
2^-133.
"""
import numpy as np
import pytest
import torch

import flow_matching_vla_euler_b200 as V
import oracle as O

pytestmark = pytest.mark.gpu


def bf16(x):
    """float64 numpy -> (bf16 CUDA tensor, its values in float64)."""
    t = torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def i32(x):
    return None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def host(t):
    t = t if t.dtype == torch.bfloat16 else t.view(torch.bfloat16)
    return t.double().cpu().numpy()


def kv_values(rng, shape):
    x = rng.standard_normal(shape) * np.exp(0.7 * rng.standard_normal(shape[-1:]))
    return x * np.exp(0.5 * rng.standard_normal(shape[:-1] + (1,)))


class Pair:
    """The cache and its model, written together."""

    def __init__(self, L, kv, D, cap, S):
        self.c = V.KVCache8(n_layers=L, n_kv_heads=kv, head_dim=D, capacity=cap, n_slots=S)
        self.m = O.Kv8Model(L, kv, D, cap, S)

    def write(self, K, V_, **kw):
        kt, kn = bf16(K)
        vt, vn = bf16(V_)
        self.c.write(kt, vt, layer=kw.get("layer", 0), **{n: i32(kw.get(n)) for n in ("pos", "count", "slots")})
        self.m.write(kn, vn, **kw)

    def check_read(self, n_tokens, fill=-3.0, **kw):
        n = kw.get("n_layers") or self.m.L - kw.get("layer", 0)
        B = kw.get("batch") or len(next(kw[x] for x in ("slots", "pos", "count") if kw.get(x) is not None))
        shape = (n, B, n_tokens, self.m.kv * self.m.D)
        k = torch.full(shape, fill, dtype=torch.bfloat16, device="cuda")
        v = torch.full(shape, fill, dtype=torch.bfloat16, device="cuda")
        dev = {x: i32(kw.get(x)) for x in ("pos", "count", "slots")}
        self.c.read(n_tokens, layer=kw.get("layer", 0), n_layers=n, batch=B, K_out=k, V_out=v, **dev)
        self.c.status()
        for w, t in ((0, k), (1, v)):
            ref = self.m.read(w, n_tokens, fill=fill, **dict(kw, batch=B))
            np.testing.assert_array_equal(host(t), ref)

    def attend(self, Q, lens, lse=True, **kw):
        qt, qn = bf16(Q)
        out = torch.full(qt.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        ls = torch.full(qt.shape[:3], 9.0, dtype=torch.float32, device="cuda") if lse else None
        dev = {x: i32(kw.get(x)) for x in ("slots", "q_pos", "q_count")}
        rest = {x: kw[x] for x in ("layer", "causal", "window", "scale") if x in kw}
        self.c.attend(qt, i32(lens), out=out, lse=ls, **dev, **rest)
        self.c.status()
        return qn, host(out), None if ls is None else ls.double().cpu().numpy()

    def check_attend(self, Q, lens, **kw):
        qn, got, ls = self.attend(Q, lens, **kw)
        ref, rls, mean_v, mag, top = self.m.attend(qn, lens, fill=7.0, **kw)
        scale = kw.get("scale") or 1.0 / np.sqrt(self.m.D)
        es = (scale * ((self.m.D + 8) * 2.0 ** -23 * mag[0] + 2.0 ** -17 * mag[1]) + 2.0 ** -20)[..., None]
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * es) * mean_v * (1 + 2.0 ** -7)
        tol += 448 * 2.0 ** -22 * top[..., None] + 2.0 ** -133
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        err = np.where(np.isnan(ref), 0.0, np.abs(got - ref) - tol)
        assert err.max() <= 0, f"err over bound {err.max():.3e}, max err {np.nanmax(np.abs(got - ref)):.3e}"
        cnt = kw.get("q_count")
        for b in range(ls.shape[0]):
            n = ls.shape[1] if cnt is None else cnt[b]
            assert np.all(ls[b, n:] == 9.0)
            a, r = ls[b, :n], rls[b, :n]
            assert np.array_equal(np.isneginf(a), np.isneginf(r)) and np.array_equal(np.isnan(a), np.isnan(r))
            ok = np.isfinite(r)
            assert np.all(np.abs(a[ok] - r[ok]) <= (es[b, :n, :, 0] + 2.0 ** -21 * np.abs(r) + 2.0 ** -20)[ok])


SHAPES = [(1, 1, 256), (2, 3, 128), (1, 2, 64), (2, 2, 32)]


# ---------------------------------------------------------------- write and read

@pytest.mark.parametrize("L,kv,D", SHAPES)
@pytest.mark.parametrize("n", [1, 63, 64, 65, 200])
def test_write_then_read(L, kv, D, n):
    rng = np.random.default_rng(n * D)
    p = Pair(L, kv, D, 211, 3)
    p.write(kv_values(rng, (L, 2, n, kv * D)), kv_values(rng, (L, 2, n, kv * D)), slots=[2, 0])
    p.check_read(n, slots=[2, 0])
    p.check_read(211, batch=3)                       # slots never written read as zeros
    if n > 5:
        p.check_read(n - 4, slots=[0, 2], pos=[3, 4], count=[n - 4, 1])


@pytest.mark.parametrize("L,kv,D", SHAPES)
def test_ragged_writes_at_odd_positions(L, kv, D):
    rng = np.random.default_rng(D)
    p = Pair(L, kv, D, 300, 4)
    p.write(kv_values(rng, (L, 4, 130, kv * D)), kv_values(rng, (L, 4, 130, kv * D)), count=[130, 1, 64, 77])
    # pieces that start inside, at the end of and past blocks; growing and shrinking magnitudes
    for step, f in enumerate((3.0, 0.01, 40.0)):
        pos = [[130, 1, 64, 77], [131, 70, 100, 78], [63, 127, 128, 5]][step]
        cnt = [[70, 69, 0, 1], [100, 1, 60, 100], [2, 65, 90, 100]][step]
        p.write(f * kv_values(rng, (L, 4, 100, kv * D)), f * kv_values(rng, (L, 4, 100, kv * D)), pos=pos, count=cnt)
        p.check_read(300, batch=4)


def test_token_by_token_equals_the_model():
    rng = np.random.default_rng(5)
    p = Pair(2, 2, 64, 140, 2)
    for t in range(140):
        f = float(np.exp(rng.standard_normal()))
        p.write(f * rng.standard_normal((2, 2, 1, 128)), f * rng.standard_normal((2, 2, 1, 128)), pos=[t, t],
                slots=[1, 0])
        if t % 23 == 0 or t == 139:
            p.check_read(t + 1, batch=2)


@pytest.mark.parametrize("L,kv,D", SHAPES)
def test_short_writes_into_growing_blocks(L, kv, D):
    """1 to 12 tokens a row (up to 8 have a kernel of their own) at odd positions, across a
    block's end, with scales that grow, shrink and stay, and a broken token in some."""
    rng = np.random.default_rng(D + 1)
    p = Pair(L, kv, D, 190, 5)
    pos = [0, 3, 60, 64, 127]
    for step, n in enumerate([1, 8, 9, 2, 5, 12, 7, 1]):
        f = [1.0, 30.0, 0.02, 500.0, 1e-3, 2e4, 1.0, 3e5][step]
        K, Vv = f * kv_values(rng, (L, 4, n, kv * D)), f * kv_values(rng, (L, 4, n, kv * D))
        if step in (2, 3, 4, 6):
            (K if step & 1 else Vv)[L - 1, step % 4, n - 1, 7] = [np.nan, np.inf][step % 2]
        slots = rng.permutation(5)[:4]
        cnt = rng.integers(0, n + 1, 4)
        cnt[step % 4] = n
        p.write(K, Vv, pos=[pos[i] for i in slots], count=cnt, slots=slots)
        for i, c in zip(slots, cnt):
            pos[i] += int(c)
        p.check_read(190, batch=5)


@pytest.mark.parametrize("L,kv,D,B,n", [(2, 8, 32, 9, 1170), (3, 2, 64, 8, 1700), (5, 3, 128, 3, 1000),
                                        (7, 2, 256, 3, 600)])
def test_writes_of_more_blocks_than_run_at_once(L, kv, D, B, n):
    """Every CTA takes several blocks in turn, some of them ragged, empty, broken or refused."""
    rng = np.random.default_rng(n)
    p = Pair(L, kv, D, n + 70, B)
    cnt = [n] * B
    cnt[1], cnt[2] = 0, n - 65
    for pos in ([0, 5, 70][:3] + [1] * (B - 3), [64, 0, 7] + [70] * (B - 3)):
        K, Vv = kv_values(rng, (L, B, n, kv * D)), kv_values(rng, (L, B, n, kv * D))
        for t in range(3, n, 97):
            (K if t & 1 else Vv)[t % L, t % B, t, t % (kv * D)] = np.nan
        p.write(K, Vv, pos=pos, count=cnt, slots=list(range(B))[::-1])
        p.check_read(n + 70, batch=B)


def test_extreme_values():
    p = Pair(1, 1, 64, 64, 1)
    x = np.zeros((1, 1, 8, 64))
    x[0, 0, 0, 0], x[0, 0, 1, 0], x[0, 0, 2, 1], x[0, 0, 3, 2] = 448.0, 1.0, 2.0 ** -9, -2.0 ** -10
    x[0, 0, 4], x[0, 0, 5, 5] = 1e-39, -447.0
    p.write(x, -x)
    p.check_read(8, batch=1)
    big = np.full((1, 1, 3, 64), 2.5e38)
    p.write(big, big, pos=[8])                       # the kept tokens fall to zero
    p.check_read(11, batch=1)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_values_that_are_not_finite(bad):
    rng = np.random.default_rng(3)
    p = Pair(1, 2, 128, 200, 1)
    K, Vv = kv_values(rng, (1, 1, 100, 256)), kv_values(rng, (1, 1, 100, 256))
    K[0, 0, 10, 5] = bad                             # head 0
    Vv[0, 0, 70, 200] = bad                          # head 1
    Vv[0, 0, 99] = bad
    p.write(K, Vv)
    p.check_read(100, batch=1)
    Q = rng.standard_normal((1, 100, 4, 128))
    p.check_attend(Q, [100], causal=True)            # rows before a broken token are not touched
    p.check_attend(Q[:, :3], [9])
    p.check_attend(Q[:, :1], [100], causal=True, window=20)
    p.write(rng.standard_normal((1, 1, 1, 256)), rng.standard_normal((1, 1, 1, 256)), pos=[64])
    p.check_attend(Q[:, :2], [65], causal=True)      # what stands behind the length does not count
    p.check_read(65, batch=1)


def test_strided_rows():
    rng = np.random.default_rng(8)
    L, B, n, kv, D = 2, 3, 70, 2, 64
    W = kv * D
    p = Pair(L, kv, D, 80, B)
    t, x = bf16(kv_values(rng, (n, L, B, 3 * W)))
    K, Vv = t[..., W:2 * W].permute(1, 2, 0, 3), t[..., 2 * W:].permute(1, 2, 0, 3)
    p.c.write(K, Vv)
    p.m.write(x[..., W:2 * W].transpose(1, 2, 0, 3), x[..., 2 * W:].transpose(1, 2, 0, 3))
    p.check_read(n, batch=B)
    o = torch.full((n, L, B, 2 * W), 5.0, dtype=torch.bfloat16, device="cuda")
    p.c.read(n, batch=B, K_out=o[..., :W].permute(1, 2, 0, 3), V_out=o[..., W:].permute(1, 2, 0, 3))
    np.testing.assert_array_equal(host(o)[..., :W].transpose(1, 2, 0, 3), p.m.read(0, n, batch=B))
    np.testing.assert_array_equal(host(o)[..., W:].transpose(1, 2, 0, 3), p.m.read(1, n, batch=B))
    # one row for every slot (stride 0 of an input)
    one, ov = bf16(kv_values(rng, (L, 1, n, W)))
    p.c.write(one.expand(L, B, n, W), one.expand(L, B, n, W))
    p.m.write(np.broadcast_to(ov, (L, B, n, W)), np.broadcast_to(ov, (L, B, n, W)))
    p.check_read(n, batch=B)


# ---------------------------------------------------------------- attention

def _filled(rng, kv, D, cap, S, L=1):
    p = Pair(L, kv, D, cap, S)
    p.write(kv_values(rng, (L, S, cap, kv * D)), kv_values(rng, (L, S, cap, kv * D)))
    return p


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 257, 700])
def test_one_token(D, n):
    rng = np.random.default_rng(D + n)
    p = _filled(rng, 2, D, n, 1)
    p.check_attend(1.5 * rng.standard_normal((1, 1, 6, D)), [n])


@pytest.mark.parametrize("group", [1, 3, 8, 16, 17, 24])
def test_groups_of_heads(group):
    rng = np.random.default_rng(group)
    p = _filled(rng, 2, 64, 150, 3)
    p.check_attend(rng.standard_normal((3, 1, 2 * group, 64)), [150, 1, 129], slots=[2, 2, 0], causal=True)


@pytest.mark.parametrize("kv,B,rows", [(4, 8, 32), (4, 8, 33), (11, 3, 32), (11, 3, 20), (1, 32, 17)])
def test_both_sides_of_the_choice_of_kernel(kv, B, rows):
    rng = np.random.default_rng(rows)
    p = _filled(rng, kv, 64, 130, B)
    lens = rng.integers(0, 131, B)
    p.check_attend(rng.standard_normal((B, rows, kv, 64)), lens, causal=True)
    p.check_attend(rng.standard_normal((B, rows, kv, 64)), lens, causal=True, window=40)


@pytest.mark.parametrize("D,kv,H,nq", [(64, 4, 20, 5), (128, 2, 8, 50), (256, 1, 8, 50), (32, 1, 4, 17), (256, 2, 2, 7),
                                       (128, 1, 3, 129), (64, 1, 1, 300)])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 37), (False, 200)])
def test_many_queries(D, kv, H, nq, causal, window):
    rng = np.random.default_rng(nq + D + window)
    p = _filled(rng, kv, D, 330, 2)
    p.check_attend(rng.standard_normal((2, nq, H, D)), [330, 303], causal=causal, window=window)


@pytest.mark.parametrize("nq", [4, 70])
def test_ragged_counts_positions_and_empty_rows(nq):
    rng = np.random.default_rng(nq)
    p = _filled(rng, 2, 128, 200, 4, L=2)
    Q = rng.standard_normal((6, nq, 8, 128))
    # lengths of zero and one, no queries, queries before the first key and behind the last
    lens, cnt = [0, 1, 200, 150, 64, 100], [nq, nq, 0, 3, 1, nq]
    pos = [0, 0, 10, -2, 63, 150]
    slots = [0, 1, 2, 3, 3, 0]
    for causal, window in ((True, 0), (True, 5), (False, 0), (False, 30)):
        p.check_attend(Q, lens, layer=1, slots=slots, q_pos=pos, q_count=cnt, causal=causal, window=window)


def test_long_row_over_many_parts():
    rng = np.random.default_rng(2)
    p = _filled(rng, 1, 64, 20000, 2)
    p.check_attend(rng.standard_normal((2, 1, 4, 64)), [20000, 77])
    p.check_attend(rng.standard_normal((2, 1, 4, 64)), [64, 19999], scale=0.5)
    p.check_attend(rng.standard_normal((2, 2, 20, 64)), [9999, 19999], causal=True, window=9000)


@pytest.mark.parametrize("D,kv,H,nq,B,window", [(256, 1, 8, 5, 1, 0), (256, 1, 8, 17, 2, 0), (128, 2, 8, 9, 1, 0),
                                                (128, 1, 4, 100, 3, 0), (64, 1, 20, 13, 1, 2500), (32, 3, 3, 65, 2, 0)])
def test_few_items_over_all_ctas(D, kv, H, nq, B, window):
    """Items whose blocks are spread over many CTAs, with a length that leaves one a single
    block and (three rows) an empty one."""
    rng = np.random.default_rng(nq)
    n = 5200
    p = _filled(rng, kv, D, n, B)
    lens = [n, 40, 0][:B]
    p.check_attend(rng.standard_normal((B, nq, H, D)), lens, causal=True, window=window)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_items_of_one_block_between_longer_ones(D):
    """One CTA after another gets items in which the second lane of the many-rows kernel has no
    block at all, and then items in which it has some: again and again, with equal bits."""
    rng = np.random.default_rng(D)
    B, nq, H = 700, 17, 2
    p = _filled(rng, 1, D, 300, 2)
    lens = np.where(np.arange(B) % 6 < 4, rng.integers(0, 65, B), rng.integers(65, 301, B))
    slots = rng.integers(0, 2, B)
    Q = rng.standard_normal((B, nq, H, D))
    p.check_attend(Q, lens, slots=slots)
    q, n, at = bf16(Q)[0], i32(lens), i32(slots)
    first = p.c.attend(q, n, slots=at)
    for _ in range(30):
        assert torch.equal(p.c.attend(q, n, slots=at), first)
    p.c.status()


def test_scores_of_unlike_size():
    """Block scales far apart, scores far apart, one key that takes all."""
    rng = np.random.default_rng(4)
    p = Pair(1, 1, 128, 400, 1)
    f = np.exp2(rng.integers(-40, 20, 7)).repeat(64)[:400, None]
    p.write(rng.standard_normal((1, 1, 400, 128)), rng.standard_normal((1, 1, 400, 128)) * f)
    Q = rng.standard_normal((1, 6, 2, 128)) * np.array([1e-30, 1e-3, 1.0, 5.0, 30.0, 1e3])[None, :, None, None]
    p.check_attend(Q, [400])
    p.check_attend(Q, [400], causal=True)
    Q[0, :, 0, 3] *= 1e4
    p.check_attend(Q, [390])
    zero = Pair(1, 1, 128, 400, 1)                   # blocks of V that are all zero
    zero.write(rng.standard_normal((1, 1, 400, 128)), np.where(f > 1, 0.0, f) * rng.standard_normal((1, 1, 400, 128)))
    zero.check_attend(Q[:, :3], [400])


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("nq", [1, 9, 70])
def test_scores_that_climb_from_block_to_block(D, nq):
    """Each block's scores pass the last one's by far (and fall back), so that every reference
    moves again and again; a row's first blocks lie outside its window."""
    rng = np.random.default_rng(D + nq)
    p = Pair(1, 1, D, 64 * 12, 2)
    f = np.repeat([1.0, 40.0, 300.0, 3.0, 2000.0, 9000.0, 0.1, 3e4, 1e5, 7.0, 2e5, 1.0], 64)
    K, Vv = (rng.standard_normal((1, 2, 64 * 12, D)) for _ in range(2))
    p.write(K * f[:, None], Vv * f[::-1, None])
    Q = rng.standard_normal((2, nq, 4, D))
    p.check_attend(Q, [64 * 12, 64 * 9 - 5])
    p.check_attend(Q, [64 * 12, 64 * 9 - 5], causal=True, window=300)


def test_strided_queries_and_outputs():
    rng = np.random.default_rng(6)
    p = _filled(rng, 2, 64, 100, 3)
    for nq in (1, 40):
        t, x = bf16(rng.standard_normal((nq, 3, 3, 8, 64)))
        q = t[:, :, 1].permute(1, 0, 2, 3)[:, :, ::2]
        buf = torch.full((nq, 4, 3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf.permute(2, 0, 1, 3)
        p.c.attend(q, i32([100, 99, 98]), causal=True, out=out)
        ref, _, mean_v, _, _ = p.m.attend(x[:, :, 1].transpose(1, 0, 2, 3)[:, :, ::2], [100, 99, 98], causal=True)
        assert np.all(np.abs(host(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7.9 * mean_v)


def test_int16_bits_are_bf16():
    rng = np.random.default_rng(7)
    p = _filled(rng, 1, 64, 40, 1)
    q, _ = bf16(rng.standard_normal((1, 3, 2, 64)))
    a = p.c.attend(q, i32([40]))
    b = p.c.attend(q.view(torch.int16), i32([40]))
    assert b.dtype == torch.int16 and torch.equal(a.view(torch.int16), b)


# ---------------------------------------------------------------- states, streams, graphs

def test_rows_out_of_range_are_left_out_and_reported():
    rng = np.random.default_rng(9)
    p = _filled(rng, 1, 64, 100, 3)
    K, _ = bf16(rng.standard_normal((1, 3, 10, 64)))
    for kw in (dict(slots=[0, 3, 1]), dict(slots=[0, -1, 1]), dict(pos=[0, 91, 0]), dict(pos=[0, -1, 0]),
               dict(count=[1, 11, 1]), dict(count=[1, -1, 1]), dict(slots=[2, 1, 2])):
        p.c.write(K, K, **{k: i32(v) for k, v in kw.items()})
        with pytest.raises(V.VlaError) as ei:
            p.c.status()
        assert ei.value.code == V.VLA_ERR_SHAPE
        p.c.status()                                  # the word was cleared
    # a refused row leaves its slot as it was
    fresh = _filled(rng, 1, 64, 100, 3)
    k, kn = bf16(rng.standard_normal((1, 3, 10, 64)))
    fresh.c.write(k, k, slots=i32([2, 7, 2]))
    fresh.m.write(kn[:, :1], kn[:, :1], slots=[2])
    with pytest.raises(V.VlaError):
        fresh.c.status()
    fresh.check_read(100, batch=3)
    for nq in (1, 60):
        q, qn = bf16(rng.standard_normal((4, nq, 2, 64)))
        out = torch.full_like(q, 7.0)
        fresh.c.attend(q, i32([100, 101, -1, 50]), slots=i32([0, 1, 2, 3]), out=out)
        with pytest.raises(V.VlaError):
            fresh.c.status()
        assert torch.all(out[1:] == 7.0)
        ref, _, mean_v, _, _ = fresh.m.attend(qn[:1], [100])
        assert np.all(np.abs(host(out[:1]) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7.9 * mean_v)


@pytest.mark.parametrize("n", [1, 8, 9])
def test_refused_rows_of_short_and_long_writes(n):
    rng = np.random.default_rng(n)
    p = _filled(rng, 2, 128, 100, 4)
    K, kn = bf16(kv_values(rng, (1, 5, n, 256)))
    # row 1 names a slot twice, row 2 one that is not there, row 4 runs over the end
    p.c.write(K, K, slots=i32([3, 3, 4, 0, 1]), pos=i32([60, 5, 0, 63, 101 - n]))
    for r, slot, pos in ((0, 3, 60), (3, 0, 63)):
        p.m.write(kn[:, r:r + 1], kn[:, r:r + 1], slots=[slot], pos=[pos])
    with pytest.raises(V.VlaError) as ei:
        p.c.status()
    assert ei.value.code == V.VLA_ERR_SHAPE
    p.check_read(60 + n, slots=[3])
    p.check_read(63 + n, slots=[0])
    p.check_read(100, slots=[1, 2])


@pytest.mark.parametrize("nq", [1, 3, 40])
@pytest.mark.parametrize("D", [64, 256])
def test_queries_that_are_not_finite_touch_their_own_rows_only(D, nq):
    rng = np.random.default_rng(nq)
    p = _filled(rng, 1, D, 300, 2)
    Q = rng.standard_normal((3, nq, 8, D))
    Q[0, 0, 2, 5], Q[1, nq - 1, 7, 0], Q[2, nq // 2, 0] = np.nan, np.inf, -np.inf
    _, got, ls = p.attend(Q, [300, 64, 300], slots=[1, 0, 1], causal=True)
    bad = np.zeros(Q.shape[:3], bool)
    bad[0, 0, 2] = bad[1, nq - 1, 7] = bad[2, nq // 2, 0] = True
    assert np.isnan(got[bad]).all() and np.isnan(ls[bad]).all()
    Q[bad] = 0.0
    _, clean, lc = p.attend(Q, [300, 64, 300], slots=[1, 0, 1], causal=True)
    assert np.array_equal(got[~bad], clean[~bad]) and np.array_equal(ls[~bad], lc[~bad])
    p.check_attend(Q, [300, 64, 300], slots=[1, 0, 1], causal=True)


def test_offsets_past_32_bits():
    """A cache of 2 x 4.6 GB, its last slot; K and V rows 2^31 elements apart."""
    rng = np.random.default_rng(1)
    D, cap, S, n = 256, 100000, 180, 70
    c = V.KVCache8(n_layers=1, n_kv_heads=1, head_dim=D, capacity=cap, n_slots=S)
    m = O.Kv8Model(1, 1, D, 2 * n, 2)
    base = torch.empty(2 ** 31 + n * D, dtype=torch.bfloat16, device="cuda")
    K = base.as_strided((1, 2, n, D), (8, 2 ** 31, D, 1))
    x, xn = bf16(kv_values(rng, (1, 2, n, D)))
    K.copy_(x)
    pos = [cap - 2 * n, 64 * 1500]
    c.write(K, K, slots=i32([S - 1, S - 2]), pos=i32(pos))
    c.write(K[:, :, :3], K[:, :, :3], slots=i32([S - 1, S - 2]), pos=i32([p + n for p in pos]))
    o, o2 = (torch.zeros_like(base).as_strided((1, 2, n, D), (8, 2 ** 31, D, 1)) for _ in range(2))
    c.read(n, slots=i32([S - 1, S - 2]), pos=i32(pos), K_out=o, V_out=o2)
    c.status()
    # the first row begins inside a block (of zeros until then), the second with one
    off = pos[0] % 64
    m.write(xn[:, :1], xn[:, :1], slots=[0], pos=[off])
    m.write(xn[:, 1:], xn[:, 1:], slots=[1])
    m.write(xn[:, :1, :3], xn[:, :1, :3], slots=[0], pos=[off + n])
    m.write(xn[:, 1:, :3], xn[:, 1:, :3], slots=[1], pos=[n])
    np.testing.assert_array_equal(host(o[0, 0]), m.read(0, n, slots=[0], pos=[off])[0, 0])
    np.testing.assert_array_equal(host(o2[0, 0]), m.read(1, n, slots=[0], pos=[off])[0, 0])
    np.testing.assert_array_equal(host(o[0, 1]), m.read(0, n, slots=[1])[0, 0])
    for nq in (1, 30):                               # the last n + 3 tokens by their window
        q, qn = bf16(rng.standard_normal((2, nq, 8, D)))
        out = c.attend(q, i32([p + n + 3 for p in pos]), slots=i32([S - 1, S - 2]), causal=True, window=n + 3 - nq)
        ref, _, mean_v, _, _ = m.attend(qn, [off + n + 3, n + 3], slots=[0, 1], causal=True, window=n + 3 - nq)
        assert np.all(np.abs(host(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -7.5 * mean_v)
    c.status()
    c.close()


def test_captured_calls_follow_the_device_arrays():
    """A captured append and attend, replayed as the positions move on; bit-identical to the
    same calls made one by one."""
    rng = np.random.default_rng(10)
    L, kv, D, H, B = 3, 2, 64, 8, 2
    start = kv_values(rng, (L, B, 60, kv * D))
    toks = kv_values(rng, (6, L, B, 1, kv * D))
    qs = rng.standard_normal((6, L, B, 1, H, D))
    eager, graph = Pair(L, kv, D, 100, B), Pair(L, kv, D, 100, B)
    for p in (eager, graph):
        p.write(start, start, count=[60, 33])
    pos, length = i32([60, 33]), i32([61, 34])
    K, _ = bf16(toks[0])
    Q, _ = bf16(qs[0])
    outs = torch.zeros((L, B, 1, H, D), dtype=torch.bfloat16, device="cuda")

    def step(c, o):
        for l in range(L):
            c.write(K[l:l + 1], K[l:l + 1], pos=pos, layer=l)
            c.attend(Q[l], length, layer=l, causal=True, out=o[l])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(graph.c, outs)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(graph.c, outs)
    ref = torch.zeros_like(outs)
    for i in range(6):
        K.copy_(bf16(toks[i])[0])
        Q.copy_(bf16(qs[i])[0])
        pos.copy_(i32([60 + i, 33 + i]))
        length.copy_(i32([61 + i, 34 + i]))
        g.replay()
        step(eager.c, ref)
        torch.cuda.synchronize()
        assert torch.equal(outs, ref), i
    graph.c.status()
    del g


@pytest.mark.parametrize("nq", [1, 40])
def test_a_call_gives_the_same_bits_again_and_on_another_stream(nq):
    rng = np.random.default_rng(11)
    p = _filled(rng, 2, 128, 3000, 3)
    q, _ = bf16(rng.standard_normal((3, nq, 8, 128)))
    lens = i32([3000, 17, 1500])
    a = p.c.attend(q, lens, causal=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = p.c.attend(q, lens, causal=True)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("D,kv,B,H", [(128, 2, 1, 8), (256, 1, 3, 8), (256, 1, 1, 16), (64, 4, 2, 8)])
def test_long_rows_from_a_cold_cache(D, kv, B, H):
    """Slow loads (every line evicted before the call) over many stages of the ring: the warps
    that share it must not overtake a stage they have no part of."""
    n = 60001
    rng = torch.Generator(device="cuda").manual_seed(D + H)
    c = V.KVCache8(n_layers=1, n_kv_heads=kv, head_dim=D, capacity=n, n_slots=B)
    x = torch.randn((1, B, n, kv * D), generator=rng, device="cuda").to(torch.bfloat16)
    c.write(x, x)
    q = torch.randn((B, 1, H, D), generator=rng, device="cuda").to(torch.bfloat16)
    lens = i32([n - 7 * b for b in range(B)])
    first = c.attend(q, lens)
    out = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.attend(q, lens, out=out)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    for _ in range(20):
        flush.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    c.status()
    del g
    k = c.read(n, batch=B)[0].view(torch.bfloat16)[0].view(B, n, kv, D)
    for b in range(B):
        m = int(lens[b])
        kb = k[b, :m].double().repeat_interleave(H // kv, dim=1)
        w = torch.softmax(torch.einsum("hd,nhd->hn", q[b, 0].double(), kb) / D ** 0.5, dim=1)
        ref = torch.einsum("hn,nhd->hd", w, kb)
        mean = torch.einsum("hn,nhd->hd", w, kb.abs())
        # the bound above with 2 e_s below 1.5e-3 (|q . k| of normal values)
        assert torch.all((first[b, 0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -7.5 * mean)


def test_tensors_of_the_host_and_wrong_types_are_refused():
    c = V.KVCache8(n_layers=1, n_kv_heads=1, head_dim=64, capacity=64, n_slots=2)
    k = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    n = torch.zeros(2, dtype=torch.int32, device="cuda")
    for call, err in [
            (lambda: c.write(k.cpu(), k), TypeError), (lambda: c.write(k.float(), k), TypeError),
            (lambda: c.write(k.half(), k), TypeError),
            (lambda: c.write(k, k[:, :, :3]), ValueError), (lambda: c.write(k, k, pos=n.long()), TypeError),
            (lambda: c.write(k, k, pos=n[:1]), ValueError), (lambda: c.write(k, k, pos=n.cpu()), TypeError),
            (lambda: c.write(k[..., :32], k[..., :32]), ValueError),
            (lambda: c.write(k[:, :, :, ::2], k), ValueError), (lambda: c.write(k, k, layer=1), V.VlaError),
            (lambda: c.write(k.new_zeros((1, 3, 4, 64)), k.new_zeros((1, 3, 4, 64))), V.VlaError),
            (lambda: c.write(k.new_zeros((1, 2, 65, 64)), k.new_zeros((1, 2, 65, 64))), V.VlaError),
            (lambda: c.write(k[:1, :1, :1, :].expand(1, 2, 4, 64), k), ValueError),
            (lambda: c.read(4, K_out=k), ValueError), (lambda: c.read(65), V.VlaError),
            (lambda: c.read(0), ValueError), (lambda: c.read(4, layer=2), ValueError),
            (lambda: c.read(4, layer=1, n_layers=1), V.VlaError),
            (lambda: c.attend(q, None), ValueError), (lambda: c.attend(q, n.cpu()), TypeError),
            (lambda: c.attend(q[..., :32], n), ValueError), (lambda: c.attend(q.float(), n), TypeError),
            (lambda: c.attend(q, n, layer=1), V.VlaError), (lambda: c.attend(q, n, window=-1), V.VlaError),
            (lambda: c.attend(q, n, scale=-1.0), ValueError), (lambda: c.attend(q, n, scale=float("inf")), V.VlaError),
            (lambda: c.attend(q, n, out=q[:1]), ValueError),
            (lambda: c.attend(q, n, lse=torch.zeros(2, 1, 4, device="cuda", dtype=torch.float64)), TypeError),
            (lambda: c.attend(q, n, out=q[:, :, :1].expand(2, 1, 4, 64)), V.VlaError)]:
        with pytest.raises(err):
            call()
    c.status()
    two = V.KVCache8(n_layers=1, n_kv_heads=2, head_dim=64, capacity=64)
    with pytest.raises(V.VlaError, match="multiple"):
        two.attend(q[:1, :, :3], n[:1])
    with pytest.raises(V.VlaError) as ei:
        V.KVCache8(n_layers=1, n_kv_heads=1, head_dim=64, capacity=1 << 30, n_slots=16)   # 2 TB
    assert ei.value.code == V.VLA_ERR_OOM
    c.read(4)                                        # the failed allocation is no other call's error
    c.status()
    c.close()
    with pytest.raises(V.VlaError):
        c.read(4)


# ---------------------------------------------------------------- together with the pipeline

def test_prefix_of_a_prefill_kept_in_the_cache_feeds_the_expert():
    """An observation's prefix goes from the prefill into a slot of the cache, is attended there,
    and comes back as the expert's prefix; the cache is the model's bit for bit, the actions are
    the oracle's on the stored values."""
    from vla_inputs import PREFILL_WORKLOADS, make_prefill_params, make_prefill_tokens
    from ._helpers import check_actions, get, make_expert, oracle_actions, run
    pwl, wl = PREFILL_WORKLOADS["prefill_tiny"], get("tiny")
    L, n, D = pwl.cfg.n_layers, pwl.n_tokens, pwl.cfg.head_dim
    pf = V.Prefill(pwl.cfg, make_prefill_params(pwl.cfg, pwl.seed), max_tokens=n)
    K, Vv = pf.run(torch.from_numpy(make_prefill_tokens(pwl)).cuda())
    p = Pair(L, 1, D, n + 3, 4)
    p.c.write(K, Vv, slots=i32([2]))
    p.m.write(host(K), host(Vv), slots=[2])
    p.check_read(n, slots=[2])
    rng = np.random.default_rng(11)
    for l in range(L):
        p.check_attend(rng.standard_normal((1, 5, wl.expert.n_heads, D)), [n], slots=[2], layer=l)
    Kb, Vb = p.c.read(n, slots=i32([2]))
    ex, inp = make_expert(wl)
    ex.set_prefix(Kb, Vb)
    got = run(ex, inp, wl.steps)
    ref = oracle_actions(wl, inp, prefix_k=Kb.cpu().numpy().view(np.uint16), prefix_v=Vb.cpu().numpy().view(np.uint16))
    check_actions(got, ref, "expert on the stored prefix")
    p.c.status()
    ex.close()
    pf.close()
