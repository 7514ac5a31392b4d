"""The 8-bit K/V cache: what is measured, in plain torch form and through the library.

Three operators share one cache of E4M3 values with a power-of-two scale for each block of
64 tokens, layer and K/V head (K and V apart):

* ``write``  stores bf16 K/V rows at given positions of given slots. A block whose earlier
  tokens are kept holds the larger of its old scale and the one the new tokens need, and
  its kept tokens are rounded again to that scale. The pass reads the touched range back,
  so the updated blocks are its outputs.
* ``read``   returns stored tokens as bf16.
* ``attend`` is softmax attention of bf16 queries over stored tokens (grouped heads,
  ragged lengths, causal and window masks).

The scale of a block is the smallest power of two s >= 2^-60 with amax / s <= 448.
"""
import math
import random

import torch

own = False

BLOCK = 64
S_MIN_EXP = -60
DEV = "cuda"


# ---------------------------------------------------------------- cases

def _write(name, L, B, kv, D, n, pos, ragged):
    """n new tokens a row at most; pos: largest position of a row's first new token."""
    return {"name": name, "op": "write", "L": L, "B": B, "kv": kv, "D": D, "n": n, "pos": pos, "ragged": ragged}


def _read(name, L, B, kv, D, n, ragged):
    return {"name": name, "op": "read", "L": L, "B": B, "kv": kv, "D": D, "n": n, "ragged": ragged}


def _attend(name, B, H, kv, D, nq, klen, ragged, causal, window):
    """klen: largest number of stored tokens of a row, the queries' own among them when causal."""
    return {"name": name, "op": "attend", "B": B, "H": H, "kv": kv, "D": D, "nq": nq, "klen": klen,
            "ragged": ragged, "causal": causal, "window": window}


def listed():
    return [
        # one observation's prefix (3 views of 256 tokens and a 20-token prompt, 18 layers) stored and read back
        _write("store_one", 18, 1, 1, 256, 788, 0, False),
        # the prefixes of 64 observations
        _write("store_batch", 18, 64, 1, 256, 788, 0, False),
        # one new token of 64 ragged sequences, all layers: the append of a control tick
        _write("append_token", 18, 64, 1, 256, 1, 851, True),
        # prompt pieces of ragged length at odd positions, several K/V heads
        _write("store_pieces", 4, 16, 8, 128, 1531, 517, True),
        # one observation's prefix back to bf16, as the expert's static region takes it
        _read("load_one", 18, 1, 1, 256, 788, False),
        # 32 ragged sequences back to bf16
        _read("load_ragged", 4, 32, 8, 128, 4096, True),
        # one query token over one observation's prefix: the smallest call
        _attend("token_one", 1, 8, 1, 256, 1, 788, False, False, 0),
        # one token of each of 64 ragged sequences
        _attend("token_batch", 64, 32, 8, 128, 1, 8192, True, True, 0),
        # one token over one long sequence
        _attend("token_long", 1, 32, 8, 128, 1, 200001, False, True, 0),
        # five tokens to be verified, window of 511 keys, odd group of heads
        _attend("verify_window", 7, 20, 4, 64, 5, 2001, True, True, 511),
        # the action chunk of 64 observations over their prefixes (no causal mask)
        _attend("chunk_batch", 64, 8, 1, 256, 50, 788, False, False, 0),
        # a prompt piece of 2048 tokens behind 4096 stored ones
        _attend("prompt_piece", 2, 32, 8, 128, 2048, 6144, False, True, 0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


_MOST_VALUES = 64 * 18 * 788 * 256       # K values of the largest listed write or read
_MOST_PAIRS = 2 * 32 * 2048 * 6144 * 128     # H * nq * klen * D of the largest listed attend
_MOST_KV = 200001 * 8 * 128 * 2              # stored K values of the largest listed attend


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend"])
    D = rng.choice([64, 128, 256])
    kv = rng.choice([1, 1, 2, 4, 8])
    if op in ("write", "read"):
        L = _log_int(rng, 1, 18)
        B = _log_int(rng, 1, 64)
        n = 1 if op == "write" and rng.random() < 0.3 else _log_int(rng, 1, 4096)
        n = max(1, min(n, _MOST_VALUES // (L * B * kv * D)))
        ragged = rng.random() < 0.6
        if op == "read":
            return {"op": op, "L": L, "B": B, "kv": kv, "D": D, "n": n, "ragged": ragged}
        pos = rng.choice([0, _log_int(rng, 1, 1000)])
        pos = max(0, min(pos, _MOST_VALUES // (L * B * kv * D) - n))
        return {"op": op, "L": L, "B": B, "kv": kv, "D": D, "n": n, "pos": pos, "ragged": ragged}
    group = rng.choice([1, 2, 3, 4, 5, 8, 8])
    H = kv * group
    causal = rng.random() < 0.6
    nq = rng.choice([1, 1, _log_int(rng, 2, 64), _log_int(rng, 2, 2048)])
    B = _log_int(rng, 1, 64)
    klen = _log_int(rng, 1, 131072 if nq == 1 else 16384)
    klen = min(klen, _MOST_KV // (B * kv * D), _MOST_PAIRS // (B * H * nq * D))
    klen = max(klen, 1)
    if causal:
        nq = min(nq, klen)
    window = rng.choice([0, 0, _log_int(rng, 1, 4096)]) if causal else 0
    return {"op": op, "B": B, "H": H, "kv": kv, "D": D, "nq": nq, "klen": klen,
            "ragged": rng.random() < 0.6, "causal": causal, "window": window}


# ---------------------------------------------------------------- inputs

def _rows(case, seed):
    """Host integers of a case: lengths and positions (the case's own, so that its work is the
    same for every seed) and slots (the seed's)."""
    B = case["B"]
    slots = list(range(B))
    random.Random(seed).shuffle(slots)
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    if case["op"] == "attend":
        low = case["nq"] if case["causal"] else 1
        lens = [rng.randint(max(low, case["klen"] // 8), case["klen"]) if case["ragged"] else case["klen"]
                for _ in range(B)]
        lens[rng.randrange(B)] = case["klen"]
        return {"slots": slots, "count": lens, "pos": [0] * B}
    n = case["n"]
    count = [rng.randint((n + 1) // 2, n) if case["ragged"] else n for _ in range(B)]
    count[rng.randrange(B)] = n
    top = case.get("pos", 0)
    pos = [rng.randint(top // 2, top) if case["ragged"] else top for _ in range(B)]
    pos[rng.randrange(B)] = top
    return {"slots": slots, "count": count, "pos": pos}


def _kv_values(gen, L, B, n, kv, D):
    """bf16 K or V: channels of unlike size and tokens of unlike norm, as projections give them."""
    x = torch.randn((L, B, n, kv * D), generator=gen, device=DEV, dtype=torch.float32)
    x *= torch.exp(0.6 * torch.randn((L, 1, 1, kv * D), generator=gen, device=DEV))
    x *= torch.exp(0.4 * torch.randn((L, B, n, 1), generator=gen, device=DEV))
    return x.to(torch.bfloat16)


def _inputs(case, seed):
    """Every array of a case, the same for the plain form, the library and the exact values."""
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)
    r = _rows(case, seed)
    B, kv, D = case["B"], case["kv"], case["D"]
    L = case.get("L", 1)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    d = {"rows": r, "slots": i32(r["slots"]), "count": i32(r["count"]), "pos": i32(r["pos"])}
    if case["op"] == "write":
        d["K"] = _kv_values(gen, L, B, case["n"], kv, D)
        d["V"] = _kv_values(gen, L, B, case["n"], kv, D)
        # tokens stored before: positions below pos
        n0 = case["pos"]
        if n0:
            d["K0"] = _kv_values(gen, L, B, n0, kv, D) * 0.7
            d["V0"] = _kv_values(gen, L, B, n0, kv, D) * 0.7
        d["count0"] = d["pos"]
        back = [p - p % BLOCK for p in r["pos"]]
        d["back_pos"] = i32(back)
        d["back_count"] = i32([p + c - q for p, c, q in zip(r["pos"], r["count"], back)])
        d["n_back"] = max(p + c - q for p, c, q in zip(r["pos"], r["count"], back))
    else:
        n0 = case["n"] if case["op"] == "read" else case["klen"]
        d["K0"] = _kv_values(gen, L, B, n0, kv, D)
        d["V0"] = _kv_values(gen, L, B, n0, kv, D)
        d["count0"] = d["count"]
        if case["op"] == "read":
            d["n_back"] = n0
        else:
            q = torch.randn((B, case["nq"], case["H"], D), generator=gen, device=DEV, dtype=torch.float32)
            d["q"] = (1.5 * q).to(torch.bfloat16)
    return d


def _capacity(case):
    return case["klen"] if case["op"] == "attend" else case["n"] + case.get("pos", 0)


def prepare(case, seed):
    d = _inputs(case, seed)
    B, kv, D = case["B"], case["kv"], case["D"]
    L = case.get("L", 1)
    st = {k: v for k, v in d.items() if k not in ("rows", "K0", "V0", "count0")}
    st["case"] = case
    if case["op"] != "attend":
        st["K_out"] = torch.zeros((L, B, d["n_back"], kv * D), dtype=torch.bfloat16, device=DEV)
        st["V_out"] = torch.zeros_like(st["K_out"])
    else:
        st["out"] = torch.zeros_like(d["q"])
    if own:
        import flow_matching_vla_euler_b200 as V
        cache = V.KVCache8(n_layers=L, n_kv_heads=kv, head_dim=D, capacity=_capacity(case), n_slots=B)
        if "K0" in d:
            cache.write(d["K0"], d["V0"], count=d["count0"], slots=d["slots"])
        st["cache"] = cache
        return st
    nb = -(-_capacity(case) // BLOCK)
    for name in ("K", "V"):
        vals = torch.zeros((L, B, nb * BLOCK, kv, D), dtype=torch.float8_e4m3fn, device=DEV)
        scale = torch.full((L, B, nb, kv), 2.0 ** S_MIN_EXP, dtype=torch.float32, device=DEV)
        if "K0" in d:
            x0 = d[name + "0"]
            for l in range(L):
                q, s, _ = _plain_window(vals[l:l + 1], scale[l:l + 1], d["slots"], torch.zeros_like(d["pos"]),
                                        d["count0"], x0[l:l + 1], kv, D)
                n = min(nb * BLOCK, q.shape[2])
                vals[l, d["slots"].long(), :n] = q[0, :, :n]
                scale[l, d["slots"].long(), :n // BLOCK] = s[0, :, :n // BLOCK]
        st["c" + name], st["s" + name] = vals, scale
    return st


# ---------------------------------------------------------------- plain forms

def _plain_window(vals, scale, slots, pos, count, x, kv, D):
    """The blocks that a write touches, after it: E4M3 values [L, B, nb * 64, kv, D], their
    scales [L, B, nb, kv], and each window token's position [B, nb * 64]."""
    L, B, n = x.shape[:3]
    nb = (n + 2 * BLOCK - 2) // BLOCK
    b0 = pos.long() // BLOCK
    t = b0[:, None] * BLOCK + torch.arange(nb * BLOCK, device=x.device)[None]
    new = (t >= pos[:, None]) & (t < (pos + count)[:, None])
    kept = t < pos[:, None]
    rows = torch.arange(B, device=x.device)[:, None]
    xn = x.view(L, B, n, kv, D)[:, rows, (t - pos[:, None]).clamp(0, n - 1)].float()
    xn = torch.where(new[None, :, :, None, None], xn, 0.0)
    sl = slots.long()[:, None]
    cap = vals.shape[2]
    blk = (b0[:, None] + torch.arange(nb, device=x.device)[None]).clamp(max=cap // BLOCK - 1)
    old_s = scale[:, sl, blk]                                              # [L, B, nb, kv]
    old = vals[:, sl, t.clamp(max=cap - 1)].float() * old_s.repeat_interleave(BLOCK, dim=2)[..., None]
    amax = xn.view(L, B, nb, BLOCK, kv, D).abs().amax(dim=(3, 5))
    m, e = torch.frexp(amax / 448.0)
    e = torch.where(m == 0.5, e - 1, e).clamp(min=S_MIN_EXP)
    s = torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, S_MIN_EXP))
    has_kept = kept.view(B, nb, BLOCK).any(dim=2)[None, :, :, None]
    s = torch.where(has_kept, torch.maximum(s, old_s), s)
    full = torch.where(kept[None, :, :, None, None], old, xn)
    q = (full / s.repeat_interleave(BLOCK, dim=2)[..., None]).to(torch.float8_e4m3fn)
    return q, s, t


def _plain_write(st):
    c = st["case"]
    kv, D = c["kv"], c["D"]
    outs = []
    for name in ("K", "V"):
        q, s, t = _plain_window(st["c" + name], st["s" + name], st["slots"], st["pos"], st["count"], st[name], kv, D)
        x = q.float() * s.repeat_interleave(BLOCK, dim=2)[..., None]
        x = torch.where((t < (st["pos"] + st["count"])[:, None])[None, :, :, None, None], x, 0.0)
        outs.append(x[:, :, :st["n_back"]].flatten(3).to(torch.bfloat16))
    return outs


def _plain_read(st):
    c = st["case"]
    n = st["n_back"]
    seen = torch.arange(n, device=st["count"].device)[None] < st["count"][:, None]
    outs = []
    for name in ("K", "V"):
        x = st["c" + name][:, st["slots"].long(), :n].float()
        s = st["s" + name][:, st["slots"].long()].repeat_interleave(BLOCK, dim=2)[:, :, :n]
        x = torch.where(seen[None, :, :, None, None], x * s[..., None], 0.0)
        outs.append(x.flatten(3).to(torch.bfloat16))
    return outs


def _plain_attend(st):
    c = st["case"]
    B, H, kv, D, nq, n = c["B"], c["H"], c["kv"], c["D"], c["nq"], c["klen"]
    G = H // kv
    sl = st["slots"].long()

    def stored(name):
        s = st["s" + name][0, sl].repeat_interleave(BLOCK, dim=1)[:, :n]
        return (st["c" + name][0, sl, :n].float() * s[..., None]).transpose(1, 2)     # [B, kv, n, D]

    q = st["q"].float().view(B, nq, kv, G, D).permute(0, 2, 1, 3, 4).reshape(B, kv, nq * G, D)
    s = (q @ stored("K").transpose(2, 3)) * (1.0 / math.sqrt(D))
    j = torch.arange(n, device=q.device)
    p = (st["count"] - nq)[:, None] + torch.arange(nq, device=q.device)[None]       # positions of the queries
    seen = (j < st["count"][:, None])[:, None].expand(B, nq, n)
    if c["causal"]:
        seen = seen & (j <= p[:, :, None])
    if c["window"]:
        seen = seen & (j > p[:, :, None] - c["window"])
    seen = seen[:, :, None].expand(B, nq, G, n).reshape(B, 1, nq * G, n)
    s = torch.where(seen, s, -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    e = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(dim=-1, keepdim=True)
    o = (e @ stored("V")) / torch.where(total > 0, total, 1.0)
    return o.view(B, kv, nq, G, D).permute(0, 2, 1, 3, 4).reshape(B, nq, H, D).to(torch.bfloat16)


def run(state):
    c = state["case"]
    if not own:
        return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[c["op"]](state)
    cache = state["cache"]
    if c["op"] == "write":
        cache.write(state["K"], state["V"], pos=state["pos"], count=state["count"], slots=state["slots"])
        return list(cache.read(state["n_back"], pos=state["back_pos"], count=state["back_count"],
                               slots=state["slots"], K_out=state["K_out"], V_out=state["V_out"]))
    if c["op"] == "read":
        return list(cache.read(state["n_back"], count=state["count"], slots=state["slots"],
                               K_out=state["K_out"], V_out=state["V_out"]))
    return cache.attend(state["q"], state["count"], slots=state["slots"], causal=c["causal"], window=c["window"],
                        out=state["out"])


# ---------------------------------------------------------------- exact values, 64 bits

def _e4m3_64(x):
    """Nearest E4M3 value of |x| <= 448, ties to even: steps of 2^(e - 3), e >= -6."""
    _, e = torch.frexp(x)
    step = torch.exp2((e.clamp(min=-5) - 4).double())
    return torch.round(x / step) * step


def _need_64(x):
    """Scale of blocks [L, blocks, tokens, kv, D]: [L, blocks, 1, kv, 1]."""
    a = x.abs().amax(dim=(2, 4), keepdim=True)
    e = torch.ceil(torch.log2(a.clamp(min=2.0 ** -80) / 448.0))
    e = torch.where(448.0 * torch.exp2(e - 1) >= a, e - 1, e)
    e = torch.where(448.0 * torch.exp2(e) < a, e + 1, e)
    return torch.exp2(e.clamp(min=float(S_MIN_EXP)))


def _store_64(x):
    """Tokens [L, n, kv, D] written from a block's start: their values, and the last block's scale."""
    L, n = x.shape[:2]
    nb = -(-n // BLOCK)
    full = x.new_zeros((L, nb * BLOCK) + tuple(x.shape[2:]))
    full[:, :n] = x
    full = full.view((L, nb, BLOCK) + tuple(x.shape[2:]))
    s = _need_64(full)
    return (_e4m3_64(full / s) * s).flatten(1, 2)[:, :n], s[:, -1]


def exact(case, seed):
    d = _inputs(case, seed)
    B, kv, D = case["B"], case["kv"], case["D"]
    L = case.get("L", 1)
    r = d["rows"]
    if case["op"] in ("write", "read"):
        outs = []
        for name in ("K", "V"):
            res = torch.zeros((L, B, d["n_back"], kv * D), dtype=torch.float64, device=DEV)
            for b in range(B):
                n0 = r["count"][b] if case["op"] == "read" else r["pos"][b]
                old, s = None, None
                if n0:
                    old, s = _store_64(d[name + "0"][:, b, :n0].double().view(L, n0, kv, D))
                if case["op"] == "read":
                    res[:, b, :n0] = old.flatten(2)
                    continue
                x = d[name][:, b, :r["count"][b]].double().view(L, -1, kv, D)
                kept = n0 % BLOCK
                parts = []
                if kept:
                    head, x = x[:, :BLOCK - kept], x[:, BLOCK - kept:]
                    s = torch.maximum(s, _need_64(head[:, None])[:, 0])
                    parts.append(_e4m3_64(torch.cat([old[:, n0 - kept:], head], dim=1) / s) * s)
                if x.shape[1]:
                    parts.append(_store_64(x)[0])
                y = torch.cat(parts, dim=1)
                res[:, b, :y.shape[1]] = y.flatten(2)
            outs.append(res)
        return outs
    H, nq = case["H"], case["nq"]
    G = H // kv
    res = torch.zeros((B, nq, H, D), dtype=torch.float64, device=DEV)
    for b in range(B):
        n = r["count"][b]
        K = _store_64(d["K0"][:, b, :n].double().view(1, n, kv, D))[0][0]
        V = _store_64(d["V0"][:, b, :n].double().view(1, n, kv, D))[0][0]
        for i0 in range(0, nq, 512):
            i1 = min(nq, i0 + 512)
            at = torch.arange(n - nq + i0, n - nq + i1, device=DEV)[:, None]
            key = torch.arange(n, device=DEV)[None]
            hide = torch.zeros((i1 - i0, n), dtype=torch.bool, device=DEV)
            if case["causal"]:
                hide |= key > at
            if case["window"]:
                hide |= key <= at - case["window"]
            for h in range(H):
                w = d["q"][b, i0:i1, h].double() @ K[:, h // G].T / math.sqrt(D)
                w = torch.softmax(w.masked_fill(hide, -math.inf), dim=1).nan_to_num(0.0)
                res[b, i0:i1, h] = w @ V[:, h // G]
    return res


# ---------------------------------------------------------------- work

def _visible(case, lens):
    """Visible (query, key) pairs of a head, and keys any query sees, over the rows."""
    pairs = keys = 0
    nq, w = case["nq"], case["window"]
    for n in lens:
        lo_first = None
        for i in range(nq):
            p = n - nq + i
            hi = min(n, p + 1) if case["causal"] else n
            lo = max(0, p - w + 1) if w else 0
            pairs += max(0, hi - lo)
            if lo_first is None:
                lo_first = lo
        keys += max(0, n - lo_first)
    return pairs, keys


def work(case):
    r = _rows(case, 0)
    B, kv, D = case["B"], case["kv"], case["D"]
    L = case.get("L", 1)
    if case["op"] == "attend":
        pairs, keys = _visible(case, r["count"])
        qo = 2 * B * case["nq"] * case["H"] * D * 2
        scales = 2 * 4 * kv * (-(-keys // BLOCK))
        return {"bytes": 2 * keys * kv * D + qo + scales, "flops": 4 * case["H"] * D * pairs}
    each = 2 * L * kv * D           # K and V values of a token
    if case["op"] == "read":
        n = sum(r["count"])
        return {"bytes": n * each * 3, "flops": n * each}
    new = sum(r["count"])
    back = sum(p % BLOCK + c for p, c in zip(r["pos"], r["count"]))
    # new rows read (2 B) and stored (1 B), the touched range read back (1 B in, 2 B out)
    return {"bytes": each * (3 * new + 3 * back), "flops": each * (2 * new + back)}
