"""The decode operators' cases: attention over the slot cache with a shared prefix, eviction by
accumulated attention weight, and matrix-vector products with 4-bit weights.

``own`` chooses between the plain forms (elementary torch operations in 32 bits) and the calls of
this package.  Shapes are Beam's (48 query / 8 KV heads of 128, hidden 5120, sliding window 512) and
those of its tensor-parallel shares.
"""
import math
import random

import torch

own = False

D = 128


def _rsn():
    import residual_stream_norm_gb300 as rsn
    return rsn


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _attn(name, B, q_len, n_q, n_kv, prefix, lo, hi, window=0, fp8=False, weights=False):
    return dict(name=name, op="attn", B=B, q_len=q_len, n_q=n_q, n_kv=n_kv, prefix=prefix, lo=lo,
                hi=hi, window=window, fp8=fp8, weights=weights)


def listed():
    return [
        # one user's chat turn on a full-attention layer: the smallest call, latency counts
        _attn("attn_b1_ctx2k", 1, 1, 48, 8, 0, 2047, 2047),
        # a sliding-window layer of a decode batch behind one system prompt, FP8 cache; the batch is
        # padded (lengths from 0)
        _attn("attn_swa512_b128_fp8", 128, 1, 48, 8, 2048, 0, 1024, window=512, fp8=True),
        # drafted tokens of 16 sequences verified at once, odd lengths
        _attn("attn_verify_b16_q4", 16, 4, 48, 8, 5001, 5, 777),
        # a decode batch of one agent's many samples behind a 32K prompt
        _attn("attn_prefix32k_b128", 128, 1, 48, 8, 32768, 1, 1024),
        # the same at ~100K context with an FP8 cache, gathering the weights that eviction goes by
        _attn("attn_prefix98k_b32_fp8_w", 32, 1, 48, 8, 98304, 100, 4096, fp8=True, weights=True),
        # long contexts that share nothing, gathering weights
        _attn("attn_ctx100k_b8_w", 8, 1, 48, 8, 0, 60000, 100000, weights=True),
        # one sequence that has just passed its budget
        dict(name="evict_b1_2k", op="evict", rows=1, width=2176, budget=2048, recent=128, lo=2049,
             hi=2049),
        # a decode batch, some sequences still below their budget
        dict(name="evict_b128_4k", op="evict", rows=128, width=4608, budget=4096, recent=511,
             lo=3000, hi=4608),
        # nine full-attention layers of eight ~100K sequences at once
        dict(name="evict_r72_100k", op="evict", rows=72, width=102400, budget=98304, recent=2048,
             lo=98305, hi=102400),
        # attention's output projection for one token
        dict(name="w4_out_t1", op="w4", T=1, N=5120, K=6144, group=128, zeros=False),
        # the merged QKV + gate projection of a small decode batch
        dict(name="w4_qkvg_t8", op="w4", T=8, N=14336, K=5120, group=64, zeros=True),
        # a dense layer's gate and up projections for a larger batch
        dict(name="w4_up_t32", op="w4", T=32, N=40960, K=5120, group=32, zeros=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "evict", "w4"])
    if op == "attn":
        while True:
            n_q, n_kv = rng.choice([(48, 8), (48, 8), (24, 4), (12, 2), (6, 1), (8, 8), (40, 8),
                                    (32, 2)])
            B = _log(rng, 1, 128)
            q_len = rng.choice([1, 1, 1, 2, 3, 4, 8])
            prefix = rng.choice([0, _log(rng, 1, 98304), _log(rng, 1000, 98304)])
            hi = _log(rng, q_len, 100000)
            lo = rng.choice([q_len, max(q_len, hi // 2), hi])
            c = _attn("", B, q_len, n_q, n_kv, prefix, lo, hi,
                      window=rng.choice([0, 0, 0, 512, rng.randint(1, 3000)]),
                      fp8=rng.random() < 0.5, weights=rng.random() < 0.3)
            del c["name"]
            rows = B * q_len * n_q
            # within the listed cases' memory and work
            if B * hi * n_kv <= 5_200_000 and rows * (prefix + hi) <= 200_000_000:
                return c
    if op == "evict":
        while True:
            rows, budget = _log(rng, 1, 512), _log(rng, 1, 98304)
            width = budget + _log(rng, 1, 4096)
            if rows * width <= 7_000_000:
                lo = rng.choice([0, budget, width])
                return dict(op="evict", rows=rows, width=width, budget=budget,
                            recent=rng.choice([0, budget, rng.randint(0, budget)]), lo=lo, hi=width)
    group = rng.choice([32, 64, 128])
    return dict(op="w4", T=_log(rng, 1, 64), N=_log(rng, 64, 20480),
                K=group * max(1, _log(rng, 256, 20480) // group), group=group,
                zeros=rng.random() < 0.5)


def _lens(case, n):
    """The ragged lengths of a case: fixed by the case, so that its work is known."""
    r = random.Random("%s %s %s" % (case["lo"], case["hi"], n))
    return [r.randint(case["lo"], case["hi"]) for _ in range(n)]


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _pages(total, gen):
    """`total` distinct slots, in runs of 16 at random places: what a paged allocator hands out."""
    pages = torch.randperm(-(-total // 16), generator=gen, device="cuda")
    return (pages[:, None] * 16 + torch.arange(16, device="cuda")).reshape(-1)


def _prepare_attn(case, gen):
    B, n_q, n_kv, P = case["B"], case["n_q"], case["n_kv"], case["prefix"]
    lens = _lens(case, B)
    width = max(1, case["hi"])
    total = P + sum(lens)
    slots = _pages(max(1, total), gen)
    num_slots = slots.numel()
    table = torch.full((B, width), -1, dtype=torch.int64, device="cuda")
    seen = torch.arange(width, device="cuda")[None] < torch.tensor(lens, device="cuda")[:, None]
    table[seen] = slots[P:total]
    # keys and values as the cache holds them; a few keys that every query leans to
    u = torch.randn((n_kv, D), generator=gen, device="cuda")
    k = torch.randn((num_slots, n_kv, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    v = torch.randn((num_slots, n_kv, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    heavy = torch.randint(0, num_slots, (1 + num_slots // 100,), generator=gen, device="cuda")
    k[heavy] = (k[heavy].float() + 0.5 * u).bfloat16()
    T = B * case["q_len"]
    qkv = torch.randn((T, n_q + 2 * n_kv, D), generator=gen, device="cuda")
    q = qkv.bfloat16()[:, :n_q]  # a view into the packed projection's rows
    q.view(T, n_kv, n_q // n_kv, D).add_((0.6 * u)[None, :, None])
    ks, vs = 1.0, 1.0
    if case["fp8"]:
        ks, vs = 0.02, 0.0125
        k = (k / ks).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v / vs).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s = dict(case=case, q=q, k=k, v=v, ks=ks, vs=vs, prefix=slots[:P].clone(), table=table,
             lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), weight=None)
    if case["weights"]:
        s["weight"] = torch.rand((B, width), generator=gen, device="cuda") * seen
    if own:
        rsn = _rsn()
        n = rsn.beam_attn_prefix_workspace(B, case["q_len"], n_q, n_kv, P, width, case["window"],
                                           case["weights"])
        s["workspace"] = torch.empty(max(1, n), dtype=torch.uint8, device="cuda")
        s["out"] = torch.empty((T, n_q, D), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((T, n_q), dtype=torch.float32, device="cuda")
        s["weight_out"] = torch.empty_like(s["weight"]) if case["weights"] else None
    return s


def _prepare_evict(case, gen):
    rows, width = case["rows"], case["width"]
    lens = torch.tensor(_lens(case, rows), dtype=torch.int32, device="cuda")
    seen = torch.arange(width, device="cuda")[None] < lens[:, None]
    table = torch.full((rows, width), -1, dtype=torch.int64, device="cuda")
    table[seen] = _pages(rows * width, gen)[:int(seen.sum())]
    # accumulated weights: most keys get little, a few much; a fifth of them exactly nothing
    w = torch.rand((rows, width), generator=gen, device="cuda")
    weight = torch.where(w < 0.2, torch.zeros_like(w), w.pow(8) * 50) * seen
    s = dict(case=case, table=table, lens=lens, weight=weight)
    if own:
        s["table_out"] = torch.empty_like(table)
        s["lens_out"] = torch.empty_like(lens)
        s["weight_out"] = torch.empty_like(weight)
        s["freed"] = torch.empty((rows, width - case["budget"]), dtype=torch.int64, device="cuda")
    return s


def _prepare_w4(case, gen):
    T, N, K, g = case["T"], case["N"], case["K"], case["group"]
    s = dict(case=case)
    s["x"] = torch.randn((T, K), generator=gen, device="cuda").bfloat16()
    s["w"] = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    s["scales"] = (0.002 + 0.01 * torch.rand((N, K // g), generator=gen, device="cuda")).bfloat16()
    s["zeros"] = torch.randint(5, 11, (N, K // g), generator=gen, device="cuda",
                               dtype=torch.uint8) if case["zeros"] else None
    if own:
        s["y"] = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"attn": _prepare_attn, "evict": _prepare_evict, "w4": _prepare_w4}[case["op"]](case, gen)


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def _rows_of(cache, slots):
    """FP32 rows of the cache at `slots` (any shape); what is held in 8 bits as its values."""
    x = cache[slots]
    return (x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x).float()


def _plain_attn(s):
    c = s["case"]
    B, L, n_q, n_kv, P, W = c["B"], c["q_len"], c["n_q"], c["n_kv"], c["prefix"], c["window"]
    G, N = n_q // n_kv, s["table"].shape[1]
    q = s["q"].float().view(B, L, n_kv, G, D).permute(2, 0, 1, 3, 4) * (s["ks"] / math.sqrt(D))
    q = q.reshape(n_kv, B * L * G, D)
    kp, vp = (_rows_of(s[x], s["prefix"]).transpose(0, 1) for x in ("k", "v"))      # [n_kv, P, D]
    at = s["table"].clamp(min=0)
    ks, vs = (_rows_of(s[x], at).permute(2, 0, 1, 3) for x in ("k", "v"))           # [n_kv, B, N, D]
    sp = (q @ kp.transpose(1, 2)).view(n_kv, B, L, G, P)
    ss = (q.view(n_kv, B, L * G, D) @ ks.transpose(2, 3)).view(n_kv, B, L, G, N)
    p = (s["lens"].long()[:, None] - L + torch.arange(L, device="cuda"))[:, :, None]  # [B, L, 1]
    jp, js = torch.arange(P, device="cuda"), torch.arange(N, device="cuda")
    seen_p = (p >= 0) & ((P + p - jp < W) | (W == 0))
    seen_s = (p >= 0) & (js <= p) & ((p - js < W) | (W == 0))
    sp.masked_fill_(~seen_p[None, :, :, None], -math.inf)
    ss.masked_fill_(~seen_s[None, :, :, None], -math.inf)
    m = ss.amax(-1, keepdim=True)
    if P:
        m = torch.maximum(m, sp.amax(-1, keepdim=True))
    m = m.clamp(min=-1e30)
    sp.sub_(m).exp_()
    ss.sub_(m).exp_()
    l = sp.sum(-1, keepdim=True) + ss.sum(-1, keepdim=True)
    o = (sp.view(n_kv, B * L * G, P) @ vp).view(n_kv, B, L, G, D)
    o += (ss.view(n_kv, B, L * G, N) @ vs).view(n_kv, B, L, G, D)
    o = torch.where(l > 0, o * s["vs"] / l, torch.zeros_like(o))
    lse = (m + l.log())[..., 0]
    out = [o.permute(1, 2, 0, 3, 4).reshape(B * L, n_q, D).bfloat16(),
           lse.permute(1, 2, 0, 3).reshape(B * L, n_q)]
    if c["weights"]:
        ss.mul_(torch.where(l > 0, 1 / l, torch.zeros_like(l)))
        out.append(s["weight"] + ss.sum((0, 2, 3)))
    return out


def _plain_evict(s):
    c = s["case"]
    rows, width = s["table"].shape
    at = torch.arange(width, device="cuda")[None]
    n = s["lens"].long()[:, None]
    over = n > c["budget"]
    old = at < n - c["recent"]
    order = torch.where(old, s["weight"], torch.full_like(s["weight"], -math.inf)).sort(
        dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, at.expand(rows, width))
    kept = (at < n) & (~over | ~old | (rank < c["budget"] - c["recent"]))
    gone = (at < n) & ~kept
    # kept entries move up in their order; what they leave is empty
    to = torch.where(kept, kept.long().cumsum(1) - 1, width)
    table = torch.full((rows, width + 1), -1, dtype=torch.int64, device="cuda")
    table.scatter_(1, to, s["table"])
    weight = torch.zeros((rows, width + 1), device="cuda").scatter_(1, to, s["weight"])
    f = width - c["budget"]
    freed = torch.full((rows, f + 1), -1, dtype=torch.int64, device="cuda")
    freed.scatter_(1, torch.where(gone, gone.long().cumsum(1) - 1, f), s["table"])
    return [table[:, :width], kept.sum(1).int(), weight[:, :width], freed[:, :f]]


def _plain_w4(s):
    c = s["case"]
    N, K, g = c["N"], c["K"], c["group"]
    q = torch.stack((s["w"] & 15, s["w"] >> 4), 2).view(N, K // g, g).float()
    q -= s["zeros"].float()[:, :, None] if c["zeros"] else 8.0
    q *= s["scales"].float()[:, :, None]
    return (s["x"].float() @ q.view(N, K).t()).bfloat16()


def run(s):
    c = s["case"]
    if not own:
        return {"attn": _plain_attn, "evict": _plain_evict, "w4": _plain_w4}[c["op"]](s)
    rsn = _rsn()
    if c["op"] == "attn":
        rsn.beam_attn_prefix_fwd(
            s["out"], s["q"], s["k"], s["v"], s["prefix"], s["table"], s["lens"], s["workspace"],
            cache_dtype=rsn.CACHE_FP8_E4M3 if c["fp8"] else rsn.CACHE_BF16, k_scale=s["ks"],
            v_scale=s["vs"], window=c["window"], lse_out=s["lse"], key_weight_in=s["weight"],
            key_weight_out=s["weight_out"])
        return [s["out"], s["lse"]] + ([s["weight_out"]] if c["weights"] else [])
    if c["op"] == "evict":
        rsn.beam_kv_evict_fwd(s["table_out"], s["lens_out"], s["weight_out"], s["freed"],
                              s["table"], s["lens"], s["weight"], c["budget"], c["recent"])
        return [s["table_out"], s["lens_out"], s["weight_out"], s["freed"]]
    rsn.beam_w4_matvec_fwd(s["y"], s["x"], s["w"], s["scales"], s["zeros"], group=c["group"])
    return s["y"]


# ---------------------------------------------------------------------------------------------
# what a pass needs, and what it should give
# ---------------------------------------------------------------------------------------------

def work(case):
    if case["op"] == "attn":
        B, L, n_q, n_kv, P, W = (case[x] for x in ("B", "q_len", "n_q", "n_kv", "prefix", "window"))
        row = 2 * n_kv * D * (1 if case["fp8"] else 2) + 8
        pairs = keys = 0
        first = P  # the first prefix key that any row sees
        for n in _lens(case, B):
            lo = n
            for p in range(max(0, n - L), n):
                below = max(0, p + 1 - W) if W else 0
                start = max(0, P + p + 1 - W) if W else 0
                pairs += p + 1 - below + max(0, P - start)
                lo, first = min(lo, below), min(first, start)
            keys += n - lo
        T = B * L
        nbytes = (P - first + keys) * row + T * n_q * (4 * D + 4)
        if case["weights"]:
            nbytes += 8 * keys
        return {"bytes": nbytes, "flops": 4 * D * n_q * pairs}
    if case["op"] == "evict":
        lens = _lens(case, case["rows"])
        kept = sum(min(n, case["budget"]) for n in lens)
        entries = case["rows"] * case["width"]
        return {"bytes": 12 * sum(lens) + 12 * entries + 8 * (entries - kept), "flops": 0}
    T, N, K, g = case["T"], case["N"], case["K"], case["group"]
    return {"bytes": N * K / 2 + N * K / g * (3 if case["zeros"] else 2) + 2 * T * (N + K),
            "flops": 2 * T * N * K}


def _exact_attn(case, s):
    """One sequence and KV head at a time, over the list of the keys that it sees."""
    L, n_q, n_kv, P, W = (case[x] for x in ("q_len", "n_q", "n_kv", "prefix", "window"))
    G = n_q // n_kv
    f8 = torch.float8_e4m3fn
    value = (lambda c, i, h: c[i, h].view(f8).double()) if case["fp8"] else (
        lambda c, i, h: c[i, h].double())
    out = torch.zeros((case["B"] * L, n_q, D), dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"] * L, n_q), -math.inf, dtype=torch.float64, device="cuda")
    weight = s["weight"].double() if case["weights"] else None
    for h in range(n_kv):
        pk, pv = value(s["k"], s["prefix"], h) * s["ks"], value(s["v"], s["prefix"], h) * s["vs"]
        for b, n in enumerate(_lens(case, case["B"])):
            sk, sv = (value(s[x], s["table"][b, :n], h) * s[y] for x, y in (("k", "ks"), ("v", "vs")))
            for i in range(max(0, L - n), L):
                end = n - L + i + 1
                lo = max(0, P + end - W) if W else 0     # of prefix and suffix in one line
                a, c = min(lo, P), max(0, lo - P)
                keys, values = torch.cat((pk[a:], sk[c:end])), torch.cat((pv[a:], sv[c:end]))
                t, hs = b * L + i, slice(h * G, h * G + G)
                z = s["q"][t, hs].double() @ keys.t() / math.sqrt(D)
                lse[t, hs] = torch.logsumexp(z, 1)
                z = torch.softmax(z, 1)
                out[t, hs] = z @ values
                if weight is not None:
                    weight[b, c:end] += z[:, P - a:].sum(0)
    return [out, lse] + ([weight] if weight is not None else [])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        if case["B"] * case["q_len"] * case["n_kv"] > 12000:
            return None
        return _exact_attn(case, s)
    if case["op"] == "evict":
        # nothing is computed but what is moved: the weights that stay, in their order
        weight = torch.zeros_like(s["weight"], dtype=torch.float64)
        for r, n in enumerate(_lens(case, case["rows"])):
            w = s["weight"][r, :n]
            if n > case["budget"]:
                old = n - case["recent"]
                best = (-w[:old]).argsort(stable=True)[:case["budget"] - case["recent"]]
                w = torch.cat((w[best.sort().values], w[old:]))
            weight[r, :w.numel()] = w
        return [None, None, weight, None]
    x, w, scales = s["x"].double(), s["w"].long(), s["scales"].double()
    y = torch.empty((case["T"], case["N"]), dtype=torch.float64, device="cuda")
    for n in range(0, case["N"], 2048):
        q = torch.empty((min(2048, case["N"] - n), case["K"]), dtype=torch.float64, device="cuda")
        q[:, 0::2], q[:, 1::2] = w[n:n + 2048] % 16, w[n:n + 2048] // 16
        z = s["zeros"][n:n + 2048].double().repeat_interleave(case["group"], 1) if case["zeros"] else 8
        y[:, n:n + 2048] = x @ ((q - z) * scales[n:n + 2048].repeat_interleave(case["group"], 1)).t()
    return y
