"""Cases of the operators of a step that checks drafted tokens: the KV cache held in 4 bits (its write and
its attention), a whole mixture-of-experts layer for a few tokens, and the verification of drafted tokens
against the target's probabilities.

``own`` chooses between the plain forms (elementary torch operations in 32 bits, in 64 where values stand
next to a border) and the calls of this package.  Shapes are Beam's (48 query / 8 KV heads of 128, hidden
5120, 256 experts of 2560, top 8 in 4 of 8 groups, sliding window 512) and those of its tensor-parallel and
expert-parallel shares; vocabularies are generic.
"""
import math
import random

import torch

own = False

D = 128
EXPERTS, GROUPS, TOPK_GROUPS, TOPK = 256, 8, 4, 8
ROUTED_SCALING = 2.5
UNIT = 2.0 ** 44          # probabilities are counted in units of 2^-44


def _rsn():
    import residual_stream_norm_gb300 as rsn
    return rsn


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def _attn(name, B, q_len, n_q, n_kv, lo, hi, group=128, window=0, n_sink=0):
    return dict(name=name, op="attn", B=B, q_len=q_len, n_q=n_q, n_kv=n_kv, lo=lo, hi=hi, group=group,
                window=window, n_sink=n_sink)


def _moe(name, T, H, F, first, local):
    return dict(name=name, op="moe", T=T, H=H, F=F, first=first, local=local)


def _verify(name, B, k, V, draft, bf16=False):
    return dict(name=name, op="verify", B=B, k=k, V=V, draft=draft, bf16=bf16)


def listed():
    return [
        # one user's chat turn on a full-attention layer: the smallest call, latency counts
        _attn("kv4_attn_b1_ctx2k", 1, 1, 48, 8, 2047, 2047),
        # a sliding-window layer of a padded decode batch (lengths from 0), the first tokens stay visible
        _attn("kv4_attn_swa512_sink4_b128", 128, 1, 48, 8, 0, 8192, window=512, n_sink=4),
        # three drafted tokens of each of 32 sequences checked at once, odd lengths, finer groups
        _attn("kv4_attn_verify_b32_q4", 32, 4, 48, 8, 5, 20001, group=64),
        # long contexts in the finest groups
        _attn("kv4_attn_ctx100k_b8_g32", 8, 1, 48, 8, 60000, 100000, group=32),
        # the tokens of a small decode step, one of them padding
        dict(name="kv4_write_t7", op="write", T=7, n_kv=8, slots=8192, group=128, skipped=1),
        # a prefill chunk of 8 sequences of 2048 tokens
        dict(name="kv4_write_t16384_g64", op="write", T=16384, n_kv=8, slots=40000, group=64, skipped=100),
        # one token on a tensor-parallel eighth of the layer: latency counts
        _moe("moe_tp8_t1", 1, 5120, 320, 0, 256),
        # two tokens' drafts on an expert-parallel eighth: full-width experts, most pairs are elsewhere
        _moe("moe_ep8_t8", 8, 5120, 2560, 96, 32),
        # a decode batch on a tensor-parallel eighth: most experts are active, some with many tokens
        _moe("moe_tp8_t64", 64, 5120, 320, 0, 256),
        # one sequence's four drafted tokens: the smallest call
        _verify("verify_b1_k4", 1, 4, 32000, True),
        # drafts without probabilities (the draft's best token each time), BF16, an odd vocabulary
        _verify("verify_b16_k3_argmax_bf16", 16, 3, 151001, False, bf16=True),
        # a large decode batch
        _verify("verify_b128_k7", 128, 7, 160000, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "write", "moe", "moe", "verify"])
    if op == "attn":
        while True:
            n_q, n_kv = rng.choice([(48, 8), (48, 8), (12, 2), (6, 1), (8, 8), (40, 8), (32, 2)])
            B, q_len = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 3, 4, 8])
            hi = _log(rng, q_len, 100000)
            lo = rng.choice([0, q_len, max(q_len, hi // 2), hi])
            c = _attn("", B, q_len, n_q, n_kv, lo, hi, group=rng.choice([32, 64, 128]),
                      window=rng.choice([0, 0, 0, 512, rng.randint(1, 3000)]),
                      n_sink=rng.choice([0, 0, 4, rng.randint(1, 100)]))
            del c["name"]
            if B * hi * n_kv <= 6_400_000 and B * q_len * n_q * hi <= 100_000_000:
                return c
    if op == "write":
        while True:
            T, n_kv = _log(rng, 1, 16384), rng.choice([1, 2, 8, 8, 5])
            slots = T + _log(rng, 1, 40000)
            if T * n_kv <= 131072:
                return dict(op="write", T=T, n_kv=n_kv, slots=slots, group=rng.choice([32, 64, 128]),
                            skipped=rng.choice([0, T // 3, 1]))
    if op == "moe":
        while True:
            local = rng.choice([256, 256, 128, 64, 32])
            H, F = 8 * _log(rng, 64, 640), 8 * _log(rng, 8, 320)
            T = _log(rng, 1, 64)
            if local * F <= 81920 and H * T * F * local <= 5120 * 64 * 320 * 256:
                c = _moe("", T, H, F, rng.choice([0, 256 - local]), local)
                del c["name"]
                return c
    while True:
        B, k, V = _log(rng, 1, 256), rng.randint(1, 12), _log(rng, 500, 200000)
        if B * (2 * k + 1) * V <= 307_200_000 and B * V <= 20_480_000:
            c = _verify("", B, k, V, rng.random() < 0.7, bf16=rng.random() < 0.4)
            del c["name"]
            return c


def _lens(case, n):
    """The ragged lengths of a case: fixed by the case, so that its work is known."""
    r = random.Random("%s %s %s" % (case["lo"], case["hi"], n))
    return [r.randint(case["lo"], case["hi"]) for _ in range(n)]


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _bf16(shape, gen, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(std)


def _prepare_attn(case, gen):
    B, n_q, n_kv, group = case["B"], case["n_q"], case["n_kv"], case["group"]
    lens = _lens(case, B)
    width, total = max(1, case["hi"]), max(1, sum(lens))
    # distinct slots in runs of 16 at random places: what a paged allocator hands out
    pages = torch.randperm(-(-total // 16), generator=gen, device="cuda")
    slots = (pages[:, None] * 16 + torch.arange(16, device="cuda")).reshape(-1)
    table = torch.full((B, width), -1, dtype=torch.int64, device="cuda")
    seen = torch.arange(width, device="cuda")[None] < torch.tensor(lens, device="cuda")[:, None]
    table[seen] = slots[:sum(lens)]
    S = slots.numel()
    # codes, and the scales and minima that keys and values of about unit variance get
    k, v = (torch.randint(0, 256, (S, n_kv, D // 2), generator=gen, device="cuda", dtype=torch.uint8)
            for _ in range(2))
    scales = []
    for _ in range(2):
        hi, lo = (1.6 + torch.rand((S, n_kv, D // group), generator=gen, device="cuda") for _ in range(2))
        scales.append(torch.stack(((hi + lo) / 15, -lo), 3).bfloat16())
    T = B * case["q_len"]
    packed = _bf16((T, n_q + 2 * n_kv, D), gen)     # a view into the packed projection's rows
    ws = None
    if own:
        n = _rsn().beam_attn_kv4_workspace(B, case["q_len"], n_q, n_kv, width, case["window"],
                                           case["n_sink"])
        ws = torch.empty(max(1, n), dtype=torch.uint8, device="cuda")
    return dict(case=case, q=packed[:, :n_q], k=k, v=v, ks=scales[0], vs=scales[1], table=table,
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), workspace=ws,
                out=torch.empty((T, n_q, D), dtype=torch.bfloat16, device="cuda"),
                lse=torch.empty((T, n_q), dtype=torch.float32, device="cuda"))


def _prepare_write(case, gen):
    T, n_kv, S = case["T"], case["n_kv"], case["slots"]
    packed = _bf16((T, 8 * n_kv, D), gen)           # K and V among a packed projection's rows
    k, v = packed[:, 6 * n_kv:7 * n_kv], packed[:, 7 * n_kv:]
    k[:, :, 5].mul_(6.0)                            # an outlier channel, as keys have them
    slot = torch.randperm(S, generator=gen, device="cuda")[:T].contiguous()
    slot[T - case["skipped"]:] = -1
    s = dict(case=case, k_in=k, v_in=v, slot=slot)
    for x in ("k", "v"):
        s[x] = torch.randint(0, 256, (S, n_kv, D // 2), generator=gen, device="cuda", dtype=torch.uint8)
        s[x + "s"] = torch.ones((S, n_kv, D // case["group"], 2), dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_moe(case, gen):
    T, H, F, E = case["T"], case["H"], case["F"], case["local"]
    ws = None
    if own:
        ws = torch.empty(_rsn().beam_moe_layer_workspace(T, H, F, E), dtype=torch.uint8, device="cuda")
    return dict(case=case, x=_bf16((T, H), gen),
                router=torch.randn((EXPERTS, H), generator=gen, device="cuda").mul_(H ** -0.5),
                bias=torch.randn(EXPERTS, generator=gen, device="cuda").mul_(0.05),
                w13=_bf16((E, 2 * F, H), gen, H ** -0.5), w2=_bf16((E, H, F), gen, F ** -0.5),
                workspace=ws, out=torch.empty((T, H), dtype=torch.bfloat16, device="cuda"),
                ids=torch.empty((T, TOPK), dtype=torch.int32, device="cuda"),
                weights=torch.empty((T, TOPK), dtype=torch.float32, device="cuda"))


def _prepare_verify(case, gen):
    B, k, V = case["B"], case["k"], case["V"]
    kind = torch.bfloat16 if case["bf16"] else torch.float32
    sharp = 2.5 if case["draft"] else 6.0
    logits = torch.randn((B, k + 1, V), generator=gen, device="cuda").mul_(sharp)
    if case["draft"]:
        u = torch.rand((B, k, V), generator=gen, device="cuda").clamp_(min=1e-12)
        tokens = (logits[:, :k] - (-u.log_()).log_()).argmax(2)
        draft = torch.softmax(logits[:, :k], 2).to(kind)
        del u
    else:
        tokens, draft = logits[:, :k].argmax(2), None
    logits.add_(torch.randn((B, k + 1, V), generator=gen, device="cuda"), alpha=0.6)
    return dict(case=case, tokens=tokens, draft=draft, target=torch.softmax(logits, 2).to(kind),
                u_accept=torch.rand((B, k), generator=gen, device="cuda"),
                u_sample=torch.rand(B, generator=gen, device="cuda"),
                out=torch.empty((B, k + 1), dtype=torch.int64, device="cuda"),
                accepted=torch.empty(B, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"attn": _prepare_attn, "write": _prepare_write, "moe": _prepare_moe,
            "verify": _prepare_verify}[case["op"]](case, gen)


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def _values(codes, scales, at):
    """FP32 values [..., n_kv, 128] that the cache's rows `at` stand for: minimum + scale * code."""
    c, s = codes[at], scales[at].float()
    x = torch.stack((c & 15, c >> 4), -1).view(*c.shape[:-1], s.shape[-2], D // s.shape[-2]).float()
    return x.mul_(s[..., :1]).add_(s[..., 1:]).flatten(-2)


def _plain_attn(s):
    c = s["case"]
    B, L, n_q, n_kv, W = c["B"], c["q_len"], c["n_q"], c["n_kv"], c["window"]
    N = s["table"].shape[1]
    at = s["table"].clamp(min=0)
    q = s["q"].float().view(B, L, n_kv, n_q // n_kv, D).permute(2, 0, 1, 3, 4) / math.sqrt(D)
    q = q.reshape(n_kv, B, -1, D)
    z = q @ _values(s["k"], s["ks"], at).permute(2, 0, 3, 1)                       # [n_kv, B, L * G, N]
    z = z.view(n_kv, B, L, n_q // n_kv, N)
    p = (s["lens"].long()[:, None] - L + torch.arange(L, device="cuda"))[:, :, None]  # [B, L, 1]
    j = torch.arange(N, device="cuda")
    seen = (p >= 0) & (j <= p) & ((p - j < W) | (j < c["n_sink"]) | (W == 0))
    z.masked_fill_(~seen[None, :, :, None], -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-1e30)
    z.sub_(m).exp_()
    l = z.sum(-1, keepdim=True)
    v = _values(s["v"], s["vs"], at).permute(2, 0, 1, 3)
    o = (z.view(n_kv, B, -1, N) @ v).view(n_kv, B, L, n_q // n_kv, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    lse = (m + l.log())[..., 0]
    return [o.permute(1, 2, 0, 3, 4).reshape(B * L, n_q, D).bfloat16(),
            lse.permute(1, 2, 0, 3).reshape(B * L, n_q)]


def _plain_write(s):
    """The cache with the tokens' rows in it: codes (equal bit for bit), scales and minima."""
    g = s["case"]["group"]
    slot = s["slot"]
    stay = slot >= 0
    out = []
    for x in ("k", "v"):
        t = s[x + "_in"][stay].float().unflatten(-1, (-1, g))
        lo = t.amin(-1, keepdim=True)
        span = t.amax(-1, keepdim=True) - lo
        scale = (span / torch.full_like(span, 15.0)).bfloat16()
        code = ((t - lo) / torch.where(scale > 0, scale, 1.0).float()).round().clamp(0, 15)
        code = torch.where(scale > 0, code, 0.0).flatten(-2).to(torch.uint8)
        codes, scales = s[x].clone(), s[x + "s"].clone()
        codes[slot[stay]] = code[..., 0::2] | code[..., 1::2] << 4
        scales[slot[stay]] = torch.cat((scale, lo.bfloat16()), -1)
        out += [codes, scales]
    return out


def _plain_moe(s):
    c = s["case"]
    T, F = c["T"], c["F"]
    # routing, in the steps of the framework's grouped top-k on FP32 logits of 64-bit sums
    z = (s["x"].double() @ s["router"].double().t()).float()
    score = 1.0 + torch.exp(-z.double()).float()
    score = torch.ones_like(score) / score
    choice = score + s["bias"]
    by_group = choice.view(T, GROUPS, -1).sort(dim=2, descending=True, stable=True).values
    group = (by_group[:, :, 0] + by_group[:, :, 1]).sort(dim=1, descending=True, stable=True).indices
    open_ = torch.zeros((T, GROUPS), dtype=torch.bool, device="cuda").scatter_(1, group[:, :TOPK_GROUPS], True)
    choice = choice.masked_fill(~open_.repeat_interleave(EXPERTS // GROUPS, 1), -math.inf)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :TOPK]
    weights = score.gather(1, ids)
    weights = weights / weights.sum(1, keepdim=True)
    # the experts of this share, one product for each (token, expert) pair
    t, slot = ((ids >= c["first"]) & (ids < c["first"] + c["local"])).nonzero(as_tuple=True)
    e = ids[t, slot] - c["first"]
    gu = torch.bmm(s["w13"][e].float(), s["x"][t].float()[:, :, None])[:, :, 0]
    h = gu[:, :F] / (1.0 + torch.exp(-gu[:, :F])) * gu[:, F:]
    y = torch.bmm(s["w2"][e].float(), h[:, :, None])[:, :, 0]
    y = y * (ROUTED_SCALING * weights[t, slot])[:, None]
    out = torch.zeros((T, TOPK, c["H"]), device="cuda").index_put_((t, slot), y).sum(1)
    return [out.bfloat16(), ids.int(), weights]


def _plain_verify(s):
    B, k, V = (s["case"][x] for x in ("B", "k", "V"))
    x = s["tokens"]
    p = s["target"][:, :k].gather(2, x[:, :, None])[:, :, 0].double()
    q = s["draft"].gather(2, x[:, :, None])[:, :, 0].double() if s["draft"] is not None else 1.0
    n = (s["u_accept"].double() * q < p).long().cumprod(1).sum(1)                  # accepted
    b, last = torch.arange(B, device="cuda"), (n - 1 + (n < k).long()).clamp(min=0)
    target = (s["target"][b, n].double().clamp(0, 1) * UNIT).round().long()
    if s["draft"] is not None:
        other = (s["draft"][b, last].double().clamp(0, 1) * UNIT).round().long()
    else:
        other = torch.zeros_like(target).scatter_(1, x[b, last][:, None], int(UNIT))
    w = torch.where((n < k)[:, None], (target - other).clamp(min=0), target)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, target)
    run_sum = w.cumsum(1)
    total = run_sum[:, -1]
    m = (s["u_sample"].double() * 2 ** 24).long()                                  # u is a multiple of 2^-24
    border = m * (total >> 24) + (m * (total & (2 ** 24 - 1)) >> 24)
    token = (run_sum <= border[:, None]).sum(1)
    token = torch.where(total > 0, token, -1)
    i = torch.arange(k + 1, device="cuda")[None]
    out = torch.cat((x, torch.full((B, 1), -1, device="cuda")), 1)
    out = torch.where(i < n[:, None], out, torch.where(i == n[:, None], token[:, None], -1))
    return [out, n.int()]


def run(s):
    c = s["case"]
    if not own:
        return {"attn": _plain_attn, "write": _plain_write, "moe": _plain_moe,
                "verify": _plain_verify}[c["op"]](s)
    rsn = _rsn()
    if c["op"] == "attn":
        rsn.beam_attn_kv4_fwd(s["out"], s["q"], s["k"], s["v"], s["ks"], s["vs"], s["table"], s["lens"],
                              s["workspace"], group=c["group"], window=c["window"], n_sink=c["n_sink"],
                              lse_out=s["lse"])
        return [s["out"], s["lse"]]
    if c["op"] == "write":
        rsn.beam_kv4_write_fwd(s["k"], s["v"], s["ks"], s["vs"], s["k_in"], s["v_in"], s["slot"],
                               group=c["group"])
        return [s["k"], s["ks"], s["v"], s["vs"]]
    if c["op"] == "moe":
        rsn.beam_moe_layer_fwd(s["out"], s["x"], s["router"], s["bias"], s["w13"], s["w2"], s["workspace"],
                               first_expert=c["first"], routed_scaling=ROUTED_SCALING,
                               topk_ids_out=s["ids"], topk_w_out=s["weights"])
        return [s["out"], s["ids"], s["weights"]]
    rsn.beam_draft_verify_fwd(s["out"], s["accepted"], s["tokens"], s["target"], s["draft"], s["u_accept"],
                              s["u_sample"])
    return [s["out"], s["accepted"]]


# ---------------------------------------------------------------------------------------------
# what a pass needs, and what it should give
# ---------------------------------------------------------------------------------------------

def work(case):
    if case["op"] == "attn":
        B, L, n_q, n_kv, W, K = (case[x] for x in ("B", "q_len", "n_q", "n_kv", "window", "n_sink"))
        row = 2 * n_kv * (D // 2 + 4 * D // case["group"]) + 8
        pairs = keys = 0
        for n in _lens(case, B):
            seen = [(max(0, p + 1 - W) if W else 0, p + 1) for p in range(max(0, n - L), n)]
            pairs += sum(end - lo + min(K, lo) for lo, end in seen)
            if seen:
                keys += n - seen[0][0] + min(K, seen[0][0])
        return {"bytes": keys * row + B * L * n_q * (4 * D + 4) + 4 * B, "flops": 4 * D * n_q * pairs}
    if case["op"] == "write":
        rows = (case["T"] - case["skipped"]) * 2 * case["n_kv"]
        return {"bytes": rows * (2 * D + D // 2 + 4 * D // case["group"]) + 8 * case["T"], "flops": 0}
    if case["op"] == "moe":
        T, H, F, E = (case[x] for x in ("T", "H", "F", "local"))
        active = E * (1 - (1 - TOPK / EXPERTS) ** T)    # expected distinct experts of this share
        return {"bytes": active * 6 * H * F + 4 * EXPERTS * (H + 1) + 4 * T * H + 8 * T * TOPK,
                "flops": T * (TOPK * E / EXPERTS * 6 * H * F + 2 * EXPERTS * H)}
    # one row of the target, and one of the drafts unless all are accepted (about 3 in 4 are, each)
    B, k, V = (case[x] for x in ("B", "k", "V"))
    rows = B * (2 - 0.75 ** k if case["draft"] else 1)
    return {"bytes": rows * V * (2 if case["bf16"] else 4), "flops": 0}


def _rows64(codes, scales, i, h):
    """[keys, 128] in 64 bits: the values of one KV head's rows."""
    c, s = codes[i, h].long(), scales[i, h].double()
    x = torch.empty((c.shape[0], D), dtype=torch.float64, device="cuda")
    x[:, 0::2], x[:, 1::2] = c % 16, c // 16
    per = D // s.shape[1]
    return s[:, :, 1].repeat_interleave(per, 1) + s[:, :, 0].repeat_interleave(per, 1) * x


def _exact_attn(case, s):
    """One sequence and KV head at a time, over the list of the keys that it sees."""
    L, n_q, n_kv, W, K = (case[x] for x in ("q_len", "n_q", "n_kv", "window", "n_sink"))
    G = n_q // n_kv
    out = torch.zeros((case["B"] * L, n_q, D), dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"] * L, n_q), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case, case["B"])):
        for i in range(max(0, L - n), L):
            end = n - L + i + 1
            lo = max(0, end - W) if W else 0
            at = torch.cat((s["table"][b, :min(K, lo)], s["table"][b, lo:end]))
            for h in range(n_kv):
                t, hs = b * L + i, slice(h * G, h * G + G)
                z = s["q"][t, hs].double() @ _rows64(s["k"], s["ks"], at, h).t() / math.sqrt(D)
                lse[t, hs] = torch.logsumexp(z, 1)
                out[t, hs] = torch.softmax(z, 1) @ _rows64(s["v"], s["vs"], at, h)
    return [out, lse]


def _exact_moe(case, s):
    H, F, first = case["H"], case["F"], case["first"]
    z = s["x"].double() @ s["router"].double().t()
    score = torch.sigmoid(z)
    choice = (score + s["bias"].double()).tolist()
    out = torch.zeros((case["T"], H), dtype=torch.float64, device="cuda")
    weights = torch.empty((case["T"], TOPK), dtype=torch.float64, device="cuda")
    users = {}
    per = EXPERTS // GROUPS
    for t, row in enumerate(choice):
        tops = [sum(sorted(row[g * per:g * per + per])[-2:]) for g in range(GROUPS)]
        best = sorted(range(GROUPS), key=lambda g: -tops[g])[:TOPK_GROUPS]
        ids = sorted((e for g in best for e in range(g * per, g * per + per)), key=lambda e: (-row[e], e))[:TOPK]
        weights[t] = score[t, ids] / score[t, ids].sum()
        for k, e in enumerate(ids):
            users.setdefault(e, []).append((t, k))
    for e, pairs in sorted(users.items()):
        if not first <= e < first + case["local"]:
            continue
        t, k = (torch.tensor(i, device="cuda") for i in zip(*pairs))
        gu = s["x"][t].double() @ s["w13"][e - first].double().t()
        g, u = gu[:, :F], gu[:, F:]
        out[t] += (g * torch.sigmoid(g) * u) @ s["w2"][e - first].double().t() * (
            ROUTED_SCALING * weights[t, k])[:, None]
    return [out, None, weights]


def exact(case, seed):
    if case["op"] == "verify":
        return None                     # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "attn":
        if case["B"] * case["q_len"] * case["n_kv"] > 8200:
            return None
        return _exact_attn(case, s)
    if case["op"] == "moe":
        return _exact_moe(case, s)
    # scales and minima, group by group; the codes are whole numbers
    got = []
    keep = s["slot"] >= 0
    for x in ("k", "v"):
        scales = s[x + "s"].double()
        t = s[x + "_in"].double()[keep].unflatten(-1, (-1, case["group"])).sort(-1).values
        scales[s["slot"][keep]] = torch.stack(((t[..., -1] - t[..., 0]) / 15, t[..., 0]), -1)
        got += [None, scales]
    return got
