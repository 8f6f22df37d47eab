"""Cases of the operators over an 8-bit paged KV cache: the quantising append, decode and
verify attention, and chunked / varlen prefill attention.

The cache holds one byte a value, e4m3 or int8, and one fp32 power-of-two scale for each
group of 16 consecutive slots of a page and kv head, K and V apart: value = code * scale.
`run` computes a case in elementary torch operations, or, where `own` is true, through the
framework's binding; `exact` computes it again from the definition in 64 bits.
"""

import math
import random

import torch

own = False

D = 128
GROUP = 16                                     # slots that share one scale
DEV = "cuda"
THETA, EPS = 1e6, 1e-6
TOP = {"e4m3": 448.0, "int8": 127.0}           # largest code
DTYPE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
MIN_EXP, MAX_EXP = -64, 63                     # range of a scale's exponent


# ------------------------------------------------------------------ cases

def _case(name, op, fmt, hq, hkv, bs, batch, new, ctx, mix=1):
    c = {"op": op, "fmt": fmt, "hq": hq, "hkv": hkv, "bs": bs, "batch": batch,
         "new_lo": new[0], "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1], "mix": mix}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step's append of a serving batch: every token lands inside a group
        # that holds earlier tokens; latency counts
        _case("append 64 decode", "append", "e4m3", 16, 8, 16, 64, (1, 1), (1, 8192)),
        # speculative verify: 5 draft tokens a sequence, runs that straddle two groups
        _case("append verify 32x5 int8", "append", "int8", 16, 8, 16, 32, (5, 5), (2048, 8192)),
        # a prefill chunk of four prompts
        _case("append 4x2048", "append", "e4m3", 16, 8, 16, 4, (2048, 2048), (0, 0)),
        # fresh prompts of mixed lengths, wide pages, 8 q heads a kv head
        _case("append ragged 16 int8", "append", "int8", 32, 4, 256, 16, (128, 2048), (0, 300)),
        # a single short sequence: latency alone
        _case("decode 1x512", "decode", "e4m3", 16, 8, 16, 1, (1, 1), (511, 511)),
        # the serving batch the decode step is sized for
        _case("decode 64x8192", "decode", "e4m3", 16, 8, 16, 64, (1, 1), (8191, 8191)),
        # few long contexts
        _case("decode 8x32768 int8", "decode", "int8", 16, 8, 64, 8, (1, 1), (32767, 32767)),
        # a batch of mixed lengths, 8 q heads a kv head
        _case("decode mixed 64", "decode", "e4m3", 32, 4, 16, 64, (1, 1), (255, 16383)),
        # speculative verify of 5 tokens a sequence
        _case("verify 32x5 int8", "decode", "int8", 16, 8, 16, 32, (5, 5), (2048, 8192)),
        # a prefill chunk of four fresh prompts
        _case("prefill 4x2048", "prefill", "e4m3", 16, 8, 16, 4, (2048, 2048), (0, 0)),
        # chunks late in long prompts: the cache is most of what is read
        _case("prefill 19x512 long", "prefill", "e4m3", 16, 8, 16, 19, (512, 512),
              (16384, 16384)),
        # fresh prompts of mixed lengths packed back to back
        _case("prefill ragged 16 int8", "prefill", "int8", 16, 8, 64, 16, (128, 2048), (0, 0)),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "decode", "prefill"))
    fmt = rng.choice(("e4m3", "int8"))
    hq, hkv = rng.choice(((16, 8), (32, 8), (32, 4), (8, 1), (12, 4), (14, 2)))
    bs = rng.choice((16, 32, 64, 96, 128, 256))
    mix = rng.randrange(1 << 20)
    if op == "append":
        kind = rng.choice(("decode", "verify", "chunk"))
        if kind == "chunk":
            batch = _log(rng, 1, 16)
            hi = _log(rng, 16, 8192 // batch)
            new = (max(1, hi // rng.choice((1, 4))), hi)
        else:
            batch = _log(rng, 1, 128)
            n = 1 if kind == "decode" else rng.randint(2, 16)
            new = (n, n)
        ctx = (0, _log(rng, 1, 16384))
    elif op == "decode":
        batch = _log(rng, 1, 128)
        n = 1 if rng.random() < 0.7 else rng.randint(2, 16)
        hi = _log(rng, 16, max(16, min(32768, 64 * 8192 * 8 // (batch * hkv) - 16)))
        new = (n, n)
        ctx = (hi if rng.random() < 0.5 else hi // rng.choice((2, 16)), hi)
    else:
        batch = _log(rng, 1, 16)
        hi = _log(rng, 2, 2048)
        # row-key pairs within the largest listed case's
        most = 19 * 16 * 512 * 16896 // 4 // (batch * hq * hi) - hi
        top = _log(rng, 1, max(1, min(16384, most)))
        new = (max(1, hi // rng.choice((1, 1, 4))), hi)
        ctx = (0 if rng.random() < 0.4 else top // 2, top)
    return _case(None, op, fmt, hq, hkv, bs, batch, new, ctx, mix)


def _lengths(case):
    """(new tokens, earlier tokens) of every sequence; they belong to the case, not the seed."""
    rng = random.Random(case["mix"])

    def pick(lo, hi):
        if lo == hi:
            return lo
        # over the logarithm where the range is wide
        return _log(rng, max(1, lo), hi) if hi > 10 * max(1, lo) else rng.randint(lo, hi)

    return [(pick(case["new_lo"], case["new_hi"]), pick(case["ctx_lo"], case["ctx_hi"]))
            for _ in range(case["batch"])]


# ----------------------------------------------------------------- inputs

def _codes(fmt, nb, bs, hkv, g):
    """Codes and scales of a cache whose values are about N(0, 1)."""
    e = (-8 if fmt == "e4m3" else -6) + torch.randint(0, 2, (nb, bs // GROUP, hkv), device=DEV,
                                                      generator=g)
    s = torch.exp2(e.float())
    x = torch.randn(nb, bs // GROUP, GROUP, hkv, D, device=DEV, generator=g)
    x = (x / s[:, :, None, :, None]).clamp_(-TOP[fmt], TOP[fmt])
    c = x.round_().to(torch.int8) if fmt == "int8" else x.to(torch.float8_e4m3fn)
    return c.view(nb, bs, hkv, D), s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    fmt, hq, hkv, bs, B = case["fmt"], case["hq"], case["hkv"], case["bs"], case["batch"]
    lens = _lengths(case)
    total = sum(n for n, _ in lens)
    st = {"case": case, "lens": lens}

    def bf16(*shape):
        return torch.randn(*shape, device=DEV, generator=g).bfloat16()

    # the append's pool holds the pages that its tokens touch, the attention's all pages
    append = case["op"] == "append"
    first = [c // bs if append else 0 for _, c in lens]
    pages = [-(-(c + n) // bs) - f for (n, c), f in zip(lens, first)]
    nb = sum(pages) + sum(pages) // 5 + 1
    perm = torch.randperm(nb, device=DEV, generator=g).to(torch.int32)
    table = torch.full((B, max(pages)), -1, dtype=torch.int32)
    starts = [0]
    for p in pages:
        starts.append(starts[-1] + p)
    order = perm.cpu()
    for b in range(B):
        table[b, :pages[b]] = order[starts[b]:starts[b + 1]]
    st["kc"], st["ks"] = _codes(fmt, nb, bs, hkv, g)
    st["vc"], st["vs"] = _codes(fmt, nb, bs, hkv, g)
    st["q"] = bf16(total, hq, D)
    # token rows: sequence and index in it
    new = torch.tensor([n for n, _ in lens])
    row_b = torch.repeat_interleave(torch.arange(B), new)
    cu = torch.zeros(B + 1, dtype=torch.int64)
    cu[1:] = torch.cumsum(new, 0)
    row_t = torch.arange(total) - cu[row_b]
    if append:
        pos = row_t + torch.tensor([c for _, c in lens])[row_b]
        page = pos // bs - torch.tensor(first)[row_b]
        st["pos"] = pos.to(DEV)
        st["slots"] = (table[row_b, page].long() * bs + pos % bs).to(DEV)
        st["k"], st["v"] = bf16(total, hkv, D), bf16(total, hkv, D)
        st["gq"], st["gk"] = ((1 + 0.2 * torch.randn(D, device=DEV, generator=g)).bfloat16()
                              for _ in range(2))
        if own:
            from paged_kv_cache_qk_gb300 import binding as lib
            st["q_out"] = torch.empty_like(st["q"])
            # the model's rotary table, built once for its longest context
            st["n_rope"] = 32768
            st["rope"] = torch.empty(lib.rope_table_bytes(st["n_rope"]), dtype=torch.uint8,
                                     device=DEV)
            lib.rope_table_build(st["rope"], st["n_rope"], THETA)
        return st
    st["table"] = table.to(DEV)
    st["seq_lens"] = (new + torch.tensor([c for _, c in lens])).to(torch.int32).to(DEV)
    st["new"] = new.to(DEV)
    st["row_b"], st["row_t"] = row_b.to(DEV), row_t.to(DEV)
    st["cu"] = cu.to(torch.int32).to(DEV)
    if own:
        from paged_kv_cache_qk_gb300 import binding as lib
        st["out"] = torch.empty(total, hq, D, dtype=torch.bfloat16, device=DEV)
        st["lse"] = torch.empty(total, hq, device=DEV)
        # the step's plan, from what the scheduler knows on the host
        st["longest"] = longest = max(n + c for n, c in lens)
        st["most_new"] = most = max(n for n, _ in lens)
        st["even"] = all(n == most for n, _ in lens)
        if case["op"] == "decode":
            st["splits"] = lib.choose_num_splits(B, hkv, most * (hq // hkv), longest,
                                                 sum(n + c for n, c in lens), bs)
            size = lib.decode_workspace_bytes(B, most, hq, D, st["splits"])
        else:
            st["splits"] = lib.choose_prefill_splits(B, hkv, most, hq // hkv, longest)
            size = lib.prefill_workspace_bytes(1, total, hq, D, st["splits"])
        st["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------ plain forms

def _quantise(y, s, fmt):
    """Codes of y against the scales s, as float values."""
    x = y / s
    return x.round() if fmt == "int8" else x.to(torch.float8_e4m3fn).float()


def _scale_exponent(amax, fmt):
    """Smallest e with amax <= TOP * 2^e, clamped; amax's exponent and significand decide."""
    m, e = torch.frexp(amax / TOP[fmt])        # amax / TOP = m 2^e, m in [0.5, 1)
    # a quotient that rounded to a power of two may lie on either side of it
    e = torch.where(amax.double() <= TOP[fmt] * torch.exp2((e - 1).double()), e - 1, e)
    return torch.where(amax > 0, e, MIN_EXP).clamp(MIN_EXP, MAX_EXP)


def _append_cache(y, codes, scales, slots, fmt, bs):
    """The cache after y [T, H, D] went into `slots`: (codes as float, scales)."""
    nb, _, H, _ = codes.shape
    gid = slots // GROUP
    n = nb * bs // GROUP
    old = scales.reshape(n, H)
    amax = torch.zeros(n, H, device=DEV).scatter_reduce(
        0, gid[:, None].expand(-1, H), y.abs().amax(-1), "amax")
    touched = torch.zeros(n, 1, device=DEV).index_fill(0, gid, 1.0) > 0
    fresh = torch.zeros(n, device=DEV).scatter_reduce(
        0, gid, (slots % GROUP == 0).float(), "amax")[:, None] > 0
    want = torch.exp2(_scale_exponent(amax, fmt).float())
    new = torch.where(touched, torch.where(fresh, want, torch.maximum(want, old)), old)
    # earlier tokens of a group whose scale grew; a group that starts anew keeps stale codes
    ratio = torch.where(touched & ~fresh, old / new, torch.ones_like(old))
    c = codes.reshape(n, GROUP, H, D).float()
    c = _quantise(c * ratio[:, None, :, None], torch.ones((), device=DEV), fmt)
    c = c.reshape(n * GROUP, H, D).index_copy(0, slots, _quantise(y, new[gid][:, :, None], fmt))
    return c.reshape(codes.shape), new.reshape(scales.shape)


def _norm_rope(x, gamma, pos):
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.float()
    inv = THETA ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
    a = pos.double()[:, None, None] * inv
    y = y.double()
    lo, hi = y[..., :D // 2], y[..., D // 2:]
    return torch.cat((lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()), -1).float()


def _append(st):
    c = st["case"]
    qh = _norm_rope(st["q"], st["gq"], st["pos"]).bfloat16()
    kc, ks = _append_cache(_norm_rope(st["k"], st["gk"], st["pos"]), st["kc"], st["ks"],
                           st["slots"], c["fmt"], c["bs"])
    vc, vs = _append_cache(st["v"].float(), st["vc"], st["vs"], st["slots"], c["fmt"], c["bs"])
    t = torch.float8_e4m3fn if c["fmt"] == "e4m3" else torch.bfloat16
    return [qh, kc.to(t), vc.to(t), ks, vs]


def _attend(st):
    c = st["case"]
    hq, hkv, bs, B = c["hq"], c["hkv"], c["bs"], c["batch"]
    G, T = hq // hkv, max(n for n, _ in st["lens"])
    ids = st["table"].long().clamp(min=0)
    P = ids.shape[1]

    def gather(codes, scales):
        x = codes[ids].view(B, P, bs // GROUP, GROUP, hkv, D).float()
        x = x * scales[ids][:, :, :, None, :, None]
        return x.view(B, P * bs, hkv, D).permute(0, 2, 1, 3)

    q = torch.zeros(B, T, hq, D, device=DEV)
    q[st["row_b"], st["row_t"]] = st["q"].float()
    q = q.view(B, T, hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * T, D)
    s = torch.matmul(q, gather(st["kc"], st["ks"]).transpose(-1, -2)) * D ** -0.5
    s = s.view(B, hkv, G, T, P * bs)
    # token t of sequence b sees the keys n < seq_len - new + t + 1
    lim = (st["seq_lens"] - st["new"])[:, None] + torch.arange(1, T + 1, device=DEV)
    hide = torch.arange(P * bs, device=DEV) >= lim[:, :, None]
    s = s.masked_fill_(hide[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, hkv, G * T, P * bs), gather(st["vc"], st["vs"]))
    o = o.view(B, hkv, G, T, D) / l
    lse = (m + l.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, hq, D)
    lse = lse.permute(0, 3, 1, 2).reshape(B, T, hq)
    return [o[st["row_b"], st["row_t"]].bfloat16(), lse[st["row_b"], st["row_t"]]]


# -------------------------------------------------------------------- run

def _run_own(st):
    from paged_kv_cache_qk_gb300 import binding as lib
    c = st["case"]
    cache = (st["kc"], st["vc"], st["ks"], st["vs"])
    if c["op"] == "append":
        lib.norm_rope_append_q8(st["q"], st["k"], st["v"], st["pos"], st["slots"], st["gq"],
                                st["gk"], THETA, EPS, *cache, q_out=st["q_out"],
                                rope_table=st["rope"], table_positions=st["n_rope"])
        # int8 codes as the numbers they are
        kc, vc = (x.bfloat16() if c["fmt"] == "int8" else x for x in (st["kc"], st["vc"]))
        return [st["q_out"], kc, vc, st["ks"], st["vs"]]
    more = {"num_splits": st["splits"], "max_seq_len_hint": st["longest"], "lse_out": st["lse"],
            "workspace": st["ws"]}
    if c["op"] == "decode":
        lib.paged_decode_q8(st["q"], *cache, st["table"], st["seq_lens"], st["out"],
                            q_len=st["most_new"], **more)
    elif st["even"]:
        lib.paged_prefill_q8(st["q"], *cache, st["table"], st["seq_lens"], st["out"],
                             q_len=st["most_new"], **more)
    else:
        lib.paged_prefill_varlen_q8(st["q"], st["cu"], st["most_new"], *cache, st["table"],
                                    st["seq_lens"], st["out"], **more)
    return [st["out"], st["lse"]]


def run(state):
    if own:
        return _run_own(state)
    return _append(state) if state["case"]["op"] == "append" else _attend(state)


# ------------------------------------------------------------------- work

def work(case):
    hq, hkv, bs = case["hq"], case["hkv"], case["bs"]
    lens = _lengths(case)
    total = sum(n for n, _ in lens)
    if case["op"] == "append":
        groups = sum(-(-(c % GROUP + n) // GROUP) for n, c in lens)
        per_token = 2 * hq * D * 2 + 2 * hkv * D * 2 + 2 * hkv * D + 16
        # norm (4 a value), rotation (3 a value), quantisation (2 a value)
        return {"bytes": total * per_token + groups * hkv * 8,
                "flops": total * D * (7 * (hq + hkv) + 4 * hkv)}
    keys = sum(n + c for n, c in lens)
    pairs = sum(n * c + n * (n + 1) // 2 for n, c in lens) * hq
    groups = sum(-(-(n + c) // GROUP) for n, c in lens)
    return {"bytes": keys * hkv * D * 2 + groups * hkv * 8 + sum(
        -(-(n + c) // bs) for n, c in lens) * 4 + total * hq * (D * 4 + 4),
            "flops": 4 * D * pairs}


# ------------------------------------------------------------------ exact

def _exact_code(x, fmt):
    """x rounded to the format, in 64 bits: to the nearest, ties to even."""
    if fmt == "int8":
        return x.round().clamp(-127, 127)
    _, e = torch.frexp(x.abs())                # |x| = m 2^e, m in [0.5, 1)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return ((x / step).round() * step).clamp(-448, 448)


def _exact_cache(y, codes, scales, slots, fmt):
    c = codes.to(torch.float32).double().view(-1, GROUP, *codes.shape[2:])
    s = scales.double().reshape(-1, scales.shape[-1])
    groups = {}
    for t, x in enumerate(slots.tolist()):
        groups.setdefault(x // GROUP, []).append((x % GROUP, t))
    for gi, members in groups.items():
        offs = torch.tensor([o for o, _ in members], device=DEV)
        rows = y[torch.tensor([t for _, t in members], device=DEV)]
        a = rows.abs().amax((0, 2))
        e = torch.ceil(torch.log2(a / TOP[fmt]).clamp(MIN_EXP - 1, MAX_EXP + 1))
        e = torch.where(a <= TOP[fmt] * torch.exp2(e - 1), e - 1, e)
        e = torch.where(a > TOP[fmt] * torch.exp2(e), e + 1, e)
        new = torch.exp2(e.clamp(MIN_EXP, MAX_EXP))
        if all(o for o, _ in members):
            new = torch.maximum(new, s[gi])
            c[gi] = _exact_code(c[gi] * (s[gi] / new)[:, None], fmt)
        s[gi] = new
        c[gi, offs] = _exact_code(rows / new[:, None], fmt)
    return c.view(codes.shape), s.view(scales.shape)


def exact(case, seed):
    st = prepare(case, seed)
    fmt, hq, hkv, bs = case["fmt"], case["hq"], case["hkv"], case["bs"]
    if case["op"] == "append":
        inv = torch.exp(-math.log(THETA) * torch.arange(64, device=DEV).double() / 64)
        turn = torch.polar(torch.ones(64, device=DEV).double(), st["pos"].double()[:, None] * inv)

        def turned(x, gamma):
            x = x.double()
            y = x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt() * gamma.double()
            z = torch.complex(y[..., :64].contiguous(), y[..., 64:].contiguous()) * turn[:, None]
            return torch.cat((z.real, z.imag), -1)

        k = _exact_cache(turned(st["k"], st["gk"]), st["kc"], st["ks"], st["slots"], fmt)
        v = _exact_cache(st["v"].double(), st["vc"], st["vs"], st["slots"], fmt)
        return [turned(st["q"], st["gq"]), k[0], v[0], k[1], v[1]]
    outs, lses = [], []
    at = 0
    for b, (n, ctx) in enumerate(st["lens"]):
        L = n + ctx
        ids = st["table"][b, :-(-L // bs)].long()
        kv = []
        for codes, scales in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
            s = scales[ids].double().repeat_interleave(GROUP, 1)
            kv.append((codes[ids].to(torch.float32).double() * s[..., None]).reshape(-1, hkv, D)[:L])
        q = st["q"][at:at + n].double()
        at += n
        seen = torch.arange(L, device=DEV) <= ctx + torch.arange(n, device=DEV)[:, None]
        o = torch.empty(n, hq, D, device=DEV, dtype=torch.float64)
        lse = torch.empty(n, hq, device=DEV, dtype=torch.float64)
        for h in range(hq):
            s = q[:, h] @ kv[0][:, h // (hq // hkv)].T / math.sqrt(D)
            s = torch.where(seen, s, -math.inf)
            lse[:, h] = torch.logsumexp(s, -1)
            o[:, h] = torch.exp(s - lse[:, h, None]) @ kv[1][:, h // (hq // hkv)]
        outs.append(o)
        lses.append(lse)
    return [torch.cat(outs), torch.cat(lses)]
