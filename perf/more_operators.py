"""Cases of four operators of a serving step over the paged bf16 cache: the append with
rotary positions of several axes, decode / verify attention and chunked / varlen prefill
attention whose scores follow rules (a tanh cap, a bias by distance, a window, documents,
a prefix), and the verdict on drafted tokens.

`run` computes a case in elementary torch operations, or, where `own` is true, through the
framework's binding; `exact` computes it again from the definition in 64 bits.
"""

import math
import random

import torch

own = False

D = 128
DEV = "cuda"
THETA, EPS = 1e6, 1e-6
POSITIONS = 32768                              # of the model's rotary table
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def _case(name, op, **more):
    c = {"op": op, **more}
    if name:
        c["name"] = name
    return c


def _append(name, hq, hkv, bs, batch, new, ctx, sections=(16, 24, 24), interleaved=False, mix=1):
    return _case(name, "append", hq=hq, hkv=hkv, bs=bs, batch=batch, new_lo=new[0], new_hi=new[1],
                 ctx_lo=ctx[0], ctx_hi=ctx[1], sec_0=sections[0], sec_1=sections[1],
                 sec_2=sections[2], interleaved=interleaved, mix=mix)


def _attention(name, op, hq, hkv, bs, batch, new, ctx, cap=0.0, slopes=False, window=0,
               documents=0, prefix=0, gain=1.0, mix=1):
    return _case(name, op, hq=hq, hkv=hkv, bs=bs, batch=batch, new_lo=new[0], new_hi=new[1],
                 ctx_lo=ctx[0], ctx_hi=ctx[1], cap=cap, slopes=slopes, window=window,
                 documents=documents, prefix=prefix, gain=gain, mix=mix)


def _drafts(name, batch, drafts, vocab, dtype, lookup=False, ragged=False, mix=1):
    return _case(name, "drafts", batch=batch, drafts=drafts, vocab=vocab, dtype=dtype,
                 lookup=lookup, ragged=ragged, mix=mix)


def listed():
    return [
        # one decode step of a serving batch of image and text prompts: latency counts
        _append("append 64 decode", 16, 8, 16, 64, (1, 1), (1, 8192)),
        # a prefill chunk of four prompts with images
        _append("append 4x2048", 16, 8, 16, 4, (2048, 2048), (0, 0)),
        # fresh prompts of mixed lengths, wide pages, the axes' frequencies interleaved
        _append("append ragged 16 interleaved", 32, 4, 256, 16, (128, 2048), (0, 300),
                sections=(24, 20, 20), interleaved=True),
        # a single short sequence of a model with capped scores: latency alone
        _attention("decode 1x512 cap", "decode", 16, 8, 16, 1, (1, 1), (511, 511), cap=50.0,
                   gain=2.0),
        # the serving batch the decode step is sized for, capped scores
        _attention("decode 64x8192 cap", "decode", 16, 8, 16, 64, (1, 1), (8191, 8191), cap=30.0,
                   gain=3.0),
        # a batch of mixed lengths, 8 q heads a kv head, a bias that falls with the distance
        _attention("decode mixed 64 distance", "decode", 32, 4, 16, 64, (1, 1), (255, 16383),
                   slopes=True),
        # speculative verify of 5 tokens a sequence in a layer that sees a window
        _attention("verify 32x5 window", "decode", 16, 8, 16, 32, (5, 5), (2048, 8192),
                   window=1024),
        # a prefill chunk of four fresh prompts, capped scores
        _attention("prefill 4x2048 cap", "prefill", 16, 8, 16, 4, (2048, 2048), (0, 0), cap=50.0,
                   gain=2.0),
        # fresh prompts packed back to back, some of them several documents, each with a
        # prefix that is read in both directions
        _attention("prefill ragged 16 documents", "prefill", 16, 8, 64, 16, (128, 2048), (0, 0),
                   documents=4, prefix=256),
        # chunks late in long prompts, in a layer that sees a window, capped scores
        _attention("prefill 19x512 window", "prefill", 16, 8, 16, 19, (512, 512), (16384, 16384),
                   cap=30.0, window=4096, gain=3.0),
        # a single sequence's drafts: latency alone
        _drafts("drafts 1x4", 1, 4, 32768, "fp32"),
        # the serving batch, a wide vocabulary
        _drafts("drafts 64x4 wide", 64, 4, 131072, "fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "decode", "prefill", "drafts"))
    hq, hkv = rng.choice(((16, 8), (32, 8), (32, 4), (8, 1), (12, 4), (14, 2)))
    bs = rng.choice((16, 32, 64, 96, 128, 256))
    mix = rng.randrange(1 << 20)
    if op == "append":
        if rng.random() < 0.5:
            batch = _log(rng, 1, 16)
            hi = _log(rng, 16, 8192 // batch)
            new = (max(1, hi // rng.choice((1, 4))), hi)
        else:
            batch, n = _log(rng, 1, 128), rng.choice((1, 1, 5))
            new = (n, n)
        a = rng.randint(8, 40)
        b = rng.randint(4, 60 - a)
        return _append(None, hq, hkv, bs, batch, new, (0, _log(rng, 1, 16384)), (a, b, 64 - a - b),
                       rng.random() < 0.5, mix)
    if op == "drafts":
        vocab, drafts = _log(rng, 1000, 150000), rng.randint(1, 12)
        batch = _log(rng, 1, max(1, min(128, 64 * 5 * 131072 // (vocab * (drafts + 1)))))
        return _drafts(None, batch, drafts, vocab, rng.choice(("fp32", "fp32", "bf16", "fp16")),
                       rng.random() < 0.3, rng.random() < 0.3, mix)
    rules = {"cap": rng.choice((0.0, 10.0, 30.0, 50.0)), "slopes": rng.random() < 0.3,
             "window": _log(rng, 1, 8192) if rng.random() < 0.4 else 0,
             "documents": rng.randint(2, 6) if rng.random() < 0.3 else 0,
             "prefix": _log(rng, 1, 2048) if rng.random() < 0.3 else 0,
             "gain": rng.choice((1.0, 2.0, 4.0)), "mix": mix}
    if op == "decode":
        batch = _log(rng, 1, 128)
        n = 1 if rng.random() < 0.7 else rng.randint(2, 16)
        hi = _log(rng, 16, max(16, min(32768, 64 * 8192 * 8 // (batch * hkv) - 16)))
        new, ctx = (n, n), (hi if rng.random() < 0.5 else hi // rng.choice((2, 16)), hi)
    else:
        batch = _log(rng, 1, 16)
        hi = _log(rng, 2, 2048)
        # row-key pairs within the largest listed case's
        most = 4 * 16 * 2048 * 4096 // (batch * hq * hi) - hi
        top = _log(rng, 1, max(1, min(16384, most)))
        new = (max(1, hi // rng.choice((1, 1, 4))), hi)
        ctx = (0 if rng.random() < 0.4 else top // 2, top)
    return _attention(None, op, hq, hkv, bs, batch, new, ctx, **rules)


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


def _starts(case, lens):
    """First key of every sequence's documents, and its prefix's length."""
    rng = random.Random(case["mix"] + 1)
    found = []
    for n, c in lens:
        cuts = sorted(rng.randrange(n + c) for _ in range(case["documents"] - 1))
        found.append(([0] + cuts, rng.randint(0, case["prefix"])))
    return found


def _axes(case):
    """Axis of each of the 64 frequencies."""
    left = [case["sec_0"], case["sec_1"], case["sec_2"]]
    if not case["interleaved"]:
        return [a for a in range(3) for _ in range(left[a])]
    axes = []
    while len(axes) < D // 2:
        for a in range(3):
            if left[a]:
                left[a] -= 1
                axes.append(a)
    return axes


# ----------------------------------------------------------------- inputs

def _image_positions(index, side):
    """Time, height and width of tokens that alternate 8 of text and an image of side x side."""
    block, o = index // (side * side + 8), index % (side * side + 8)
    base = block * (side + 8)
    at = (o - 8).clamp(min=0)
    text = o < 8
    start = torch.where(text, base + o, base + 8)
    return torch.stack((start, torch.where(text, start, start + at // side),
                        torch.where(text, start, start + at % side)))


def _prepare_drafts(case, g):
    B, K, V, dtype = case["batch"], case["drafts"], case["vocab"], TYPES[case["dtype"]]
    rng = random.Random(case["mix"])
    # a peaked target, and a draft model near it
    logits = 3.0 * torch.randn(B, K + 1, V, device=DEV, generator=g)
    st = {"case": case, "p": torch.softmax(logits, -1).to(dtype)}
    near = logits[:, :K] + 0.7 * torch.randn(B, K, V, device=DEV, generator=g)
    q = torch.softmax(near, -1)
    # drafted tokens: drawn from the draft model, or (looked up in the prompt) its likeliest
    if case["lookup"]:
        st["q"], drafts = None, q.argmax(-1)
    else:
        st["q"] = q.to(dtype)
        u = torch.rand(B, K, 1, device=DEV, generator=g, dtype=torch.float64)
        c = st["q"].double().cumsum(-1)
        drafts = torch.searchsorted(c, u * c[..., -1:], right=True)[..., 0].clamp(max=V - 1)
    st["drafts"] = drafts.to(torch.int32).contiguous()
    st["u"] = torch.rand(B, K + 1, device=DEV, generator=g)
    lens = [rng.randint(0, K) if case["ragged"] else K for _ in range(B)]
    st["draft_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["seq_lens"] = torch.tensor([rng.randint(1, 8192) + n + 1 for n in lens], dtype=torch.int32,
                                  device=DEV)
    if own:
        st["tokens"] = torch.empty(B, K + 1, dtype=torch.int32, device=DEV)
        st["accepted"] = torch.empty(B, dtype=torch.int32, device=DEV)
        st["kept"] = torch.empty(B, dtype=torch.int32, device=DEV)
    return st


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] == "drafts":
        return _prepare_drafts(case, g)
    hq, hkv, bs, B = case["hq"], case["hkv"], case["bs"], case["batch"]
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
    order = torch.randperm(nb, device=DEV, generator=g).to(torch.int32).cpu()
    table = torch.full((B, max(pages)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    st["kc"], st["vc"] = bf16(nb, bs, hkv, D), bf16(nb, bs, hkv, D)
    st["q"] = bf16(total, hq, D)
    # token rows: sequence and index in it
    new = torch.tensor([n for n, _ in lens])
    ctx = torch.tensor([c for _, c in lens])
    row_b = torch.repeat_interleave(torch.arange(B), new)
    cu = torch.zeros(B + 1, dtype=torch.int64)
    cu[1:] = torch.cumsum(new, 0)
    row_t = torch.arange(total) - cu[row_b]
    index = row_t + ctx[row_b]
    if append:
        rng = random.Random(case["mix"] + 2)
        side = torch.tensor([rng.randint(8, 32) for _ in range(B)])[row_b]
        st["pos"] = _image_positions(index, side).contiguous().to(DEV)
        page = index // bs - torch.tensor(first)[row_b]
        st["slots"] = (table[row_b, page].long() * bs + index % bs).to(DEV)
        st["k"], st["v"] = bf16(total, hkv, D), bf16(total, hkv, D)
        st["gq"], st["gk"] = ((1 + 0.2 * torch.randn(D, device=DEV, generator=g)).bfloat16()
                              for _ in range(2))
        st["axes"] = torch.tensor(_axes(case), device=DEV)
        if own:
            from paged_kv_cache_qk_gb300 import binding as lib
            st["q_out"] = torch.empty_like(st["q"])
            # the model's rotary table, built once for its longest context
            st["rope"] = torch.empty(lib.rope_table_bytes(POSITIONS), dtype=torch.uint8,
                                     device=DEV)
            lib.rope_table_build(st["rope"], POSITIONS, THETA)
            st["freq_axes"] = lib.rope_axes((case["sec_0"], case["sec_1"], case["sec_2"]),
                                            interleaved=case["interleaved"])
        return st
    st["q"] = (st["q"].float() * case["gain"]).bfloat16()
    st["table"] = table.to(DEV)
    st["seq_lens"] = (new + ctx).to(torch.int32).to(DEV)
    st["new"] = new.to(DEV)
    st["row_b"], st["row_t"] = row_b.to(DEV), row_t.to(DEV)
    st["cu"] = cu.to(torch.int32).to(DEV)
    # a slope for each q head, falling by powers of two over the heads
    st["slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device=DEV) / hq) \
        if case["slopes"] else None
    starts = _starts(case, lens)
    st["prefix"] = torch.tensor([p for _, p in starts], dtype=torch.int32, device=DEV) \
        if case["prefix"] else None
    st["first"] = None
    if case["documents"]:
        # each row's document: the last that starts at or before its position
        begin = torch.tensor([d for d, _ in starts])[row_b]
        begin = torch.where(begin <= index[:, None], begin, 0).amax(1)
        st["first"] = begin.to(torch.int32).to(DEV)
    if own:
        from paged_kv_cache_qk_gb300 import binding as lib
        st["out"] = torch.empty(total, hq, D, dtype=torch.bfloat16, device=DEV)
        st["lse"] = torch.empty(total, hq, device=DEV)
        # the step's plan, from what the scheduler knows on the host: the keys from a
        # sequence's first visible one to its end
        st["most_new"] = most = max(n for n, _ in lens)
        st["even"] = all(n == most for n, _ in lens)
        reach = case["window"] + most - 1 if case["window"] else 1 << 30
        spans = [min(n + c, reach) for n, c in lens]
        st["longest"] = longest = max(spans)
        if case["op"] == "decode":
            st["splits"] = lib.choose_num_splits(B, hkv, most * (hq // hkv), longest, sum(spans),
                                                 bs)
            size = lib.decode_workspace_bytes(B, most, hq, D, st["splits"])
        else:
            st["splits"] = lib.choose_prefill_splits(B, hkv, most, hq // hkv, longest)
            size = lib.prefill_workspace_bytes(1, total, hq, D, st["splits"])
        st["ws"] = torch.empty(max(size, 256), dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------ plain forms

def _plain_append(st):
    c = st["case"]
    inv = THETA ** (-torch.arange(0, D, 2, device=DEV, dtype=torch.float64) / D)
    # the position of a frequency is that of its axis
    a = (st["pos"][st["axes"]].T.double() * inv)[:, None]

    def turned(x, gamma):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * gamma.float()
        lo, hi = y[..., :D // 2].double(), y[..., D // 2:].double()
        return torch.cat((lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()), -1).bfloat16()

    rows = st["kc"].shape[0] * c["bs"]
    kc = st["kc"].view(rows, c["hkv"], D).index_copy(0, st["slots"], turned(st["k"], st["gk"]))
    vc = st["vc"].view(rows, c["hkv"], D).index_copy(0, st["slots"], st["v"])
    return [turned(st["q"], st["gq"]), kc.view_as(st["kc"]), vc.view_as(st["vc"])]


def _plain_attention(st):
    c = st["case"]
    hq, hkv, bs, B = c["hq"], c["hkv"], c["bs"], c["batch"]
    G, T = hq // hkv, max(n for n, _ in st["lens"])
    ids = st["table"].long().clamp(min=0)
    P = ids.shape[1]

    def gather(x):
        return x[ids].view(B, P * bs, hkv, D).permute(0, 2, 1, 3).float()

    q = torch.zeros(B, T, hq, D, device=DEV)
    q[st["row_b"], st["row_t"]] = st["q"].float()
    q = q.view(B, T, hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * T, D)
    s = torch.matmul(q, gather(st["kc"]).transpose(-1, -2)).mul_(D ** -0.5)
    s = s.view(B, hkv, G, T, P * bs)
    if c["cap"]:
        s = s.div_(c["cap"]).tanh_().mul_(c["cap"])
    # token t of sequence b sits at position seq_len - new + t
    pos = (st["seq_lens"] - st["new"])[:, None] + torch.arange(T, device=DEV)
    key = torch.arange(P * bs, device=DEV)
    if c["slopes"]:
        far = (pos[:, :, None] - key).abs().float()
        s = s.addcmul_(st["slopes"].view(1, hkv, G, 1, 1), far[:, None, None], value=-1.0)
    end = pos + 1
    if st["prefix"] is not None:
        end = torch.maximum(end, torch.minimum(st["prefix"], st["seq_lens"])[:, None])
    begin = torch.zeros_like(pos)
    if c["window"]:
        begin = (pos - c["window"] + 1).clamp(min=0)
    if st["first"] is not None:
        doc = torch.zeros(B, T, dtype=torch.int32, device=DEV)
        doc[st["row_b"], st["row_t"]] = st["first"]
        begin = torch.maximum(begin, doc)
    hide = (key < begin[:, :, None]) | (key >= end[:, :, None])
    s = s.masked_fill_(hide[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m.clamp(min=-3e38)).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, hkv, G * T, P * bs), gather(st["vc"]))
    # a row that sees no key is 0 and -inf
    o = o.view(B, hkv, G, T, D) / torch.where(l > 0, l, 1.0)
    lse = (m + l.log()).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, hq, D)
    lse = lse.permute(0, 3, 1, 2).reshape(B, T, hq)
    return [o[st["row_b"], st["row_t"]].bfloat16(), lse[st["row_b"], st["row_t"]]]


def _plain_drafts(st):
    c = st["case"]
    B, K, V = c["batch"], c["drafts"], c["vocab"]
    x = st["drafts"].long()[..., None]
    n = st["draft_lens"].long()
    at = torch.arange(K, device=DEV)
    px = st["p"][:, :K].gather(-1, x)[..., 0].double()
    qx = torch.ones_like(px) if st["q"] is None else st["q"].gather(-1, x)[..., 0].double()
    good = (st["u"][:, :K].double() * qx < px) & (at < n[:, None])
    j = good.long().cumprod(-1).sum(-1)        # drafts accepted
    seq = torch.arange(B, device=DEV)
    p = st["p"][seq, j].double()
    refused = (j < n)[:, None]
    jq = j.clamp(max=K - 1)
    if st["q"] is None:
        other = torch.zeros_like(p).scatter_(-1, x[seq, jq], 1.0)
    else:
        other = st["q"][seq, jq].double()
    w = torch.where(refused, (p - other).clamp(min=0), p)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, p)
    cum = w.cumsum(-1)
    t = st["u"][:, K:].double() * cum[:, -1:]
    token = (cum <= t).sum(-1).clamp(max=V - 1)
    pos = torch.arange(K + 1, device=DEV)
    wide = torch.cat((st["drafts"], st["drafts"][:, :1]), 1).long()
    tokens = torch.where(pos < j[:, None], wide, -1)
    tokens = torch.where(pos == j[:, None], token[:, None], tokens)
    return [tokens.int(), j.int(), (st["seq_lens"] - (n - j)).int()]


# -------------------------------------------------------------------- run

def _run_own(st):
    from paged_kv_cache_qk_gb300 import binding as lib
    c = st["case"]
    if c["op"] == "append":
        lib.norm_rope_append_axes(st["q"], st["k"], st["v"], st["pos"], st["freq_axes"],
                                  st["slots"], st["gq"], st["gk"], THETA, EPS, st["kc"], st["vc"],
                                  q_out=st["q_out"], rope_table=st["rope"],
                                  table_positions=POSITIONS)
        return [st["q_out"], st["kc"], st["vc"]]
    if c["op"] == "drafts":
        lib.verify_drafts(st["p"], st["q"], st["drafts"], st["u"], st["tokens"], st["accepted"],
                          draft_lens=st["draft_lens"], seq_lens=st["seq_lens"],
                          kept_lens=st["kept"])
        return [st["tokens"], st["accepted"], st["kept"]]
    rules = {"softcap": c["cap"], "window": c["window"], "slopes": st["slopes"],
             "first_keys": st["first"], "prefix_lens": st["prefix"]}
    more = {"num_splits": st["splits"], "max_seq_len_hint": st["longest"], "lse_out": st["lse"],
            "workspace": st["ws"]}
    if c["op"] == "decode":
        lib.paged_decode_scored(st["q"], st["kc"], st["vc"], st["table"], st["seq_lens"],
                                st["out"], q_len=st["most_new"], **rules, **more)
    elif st["even"]:
        lib.paged_prefill_scored(st["q"], st["kc"], st["vc"], st["table"], st["seq_lens"],
                                 st["out"], q_len=st["most_new"], **rules, **more)
    else:
        lib.paged_prefill_varlen_scored(st["q"], st["cu"], st["most_new"], st["kc"], st["vc"],
                                        st["table"], st["seq_lens"], st["out"], **rules, **more)
    return [st["out"], st["lse"]]


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    return {"append": _plain_append, "drafts": _plain_drafts}.get(op, _plain_attention)(state)


# ------------------------------------------------------------------- work

def work(case):
    if case["op"] == "drafts":
        B, K, V = case["batch"], case["drafts"], case["vocab"]
        size = 4 if case["dtype"] == "fp32" else 2
        # one row of each model's probabilities a sequence (which one, its drafts decide)
        rows = 1 if case["lookup"] else 2
        return {"bytes": B * (rows * V * size + K * (4 + 2 * size) + (K + 1) * 8 + 20),
                "flops": B * V * (2 + rows)}
    hq, hkv, bs = case["hq"], case["hkv"], case["bs"]
    lens = _lengths(case)
    total = sum(n for n, _ in lens)
    if case["op"] == "append":
        per_token = 2 * hq * D * 2 + 4 * hkv * D * 2 + 32
        # norm (4 a value), rotation (3 a value)
        return {"bytes": total * per_token, "flops": total * D * 7 * (hq + hkv)}
    keys = pairs = pages = 0
    for (n, c), (cuts, prefix) in zip(lens, _starts(case, lens)):
        low = n + c
        for p in range(c, c + n):
            end = max(p + 1, min(prefix, n + c))
            begin = max(p - case["window"] + 1, 0) if case["window"] else 0
            if case["documents"]:
                begin = max(begin, max(d for d in cuts if d <= p))
            low = min(low, begin)
            pairs += max(0, end - begin)
        keys += n + c - low
        pages += -(-(n + c) // bs) - low // bs
    return {"bytes": keys * hkv * D * 4 + pages * 4 + total * hq * (D * 4 + 4),
            "flops": 4 * D * hq * pairs}


# ------------------------------------------------------------------ exact

def _exact_append(st):
    c = st["case"]
    T = st["q"].shape[0]
    inv = torch.exp(-math.log(THETA) * torch.arange(64, device=DEV).double() / 64)
    at = torch.empty(T, 64, device=DEV, dtype=torch.float64)
    for i, axis in enumerate(_axes(c)):
        at[:, i] = st["pos"][axis].double() * inv[i]
    turn = torch.polar(torch.ones_like(at), at)[:, None]

    def turned(x, gamma):
        x = x.double()
        y = x / (x.square().sum(-1, keepdim=True) / D + EPS).sqrt() * gamma.double()
        z = torch.complex(y[..., :64].contiguous(), y[..., 64:].contiguous()) * turn
        return torch.cat((z.real, z.imag), -1)

    caches = []
    for cache, x in ((st["kc"], turned(st["k"], st["gk"])), (st["vc"], st["v"].double())):
        new = cache.double()
        new[st["slots"] // c["bs"], st["slots"] % c["bs"]] = x
        caches.append(new)
    return [turned(st["q"], st["gq"])] + caches


def _exact_attention(st):
    c = st["case"]
    hq, hkv, bs = c["hq"], c["hkv"], c["bs"]
    outs, lses = [], []
    at = 0
    for b, ((n, ctx), (cuts, prefix)) in enumerate(zip(st["lens"], _starts(c, st["lens"]))):
        L = n + ctx
        ids = st["table"][b, :-(-L // bs)].long()
        k, v = (x[ids].double().reshape(-1, hkv, D)[:L] for x in (st["kc"], st["vc"]))
        q = st["q"][at:at + n].double()
        at += n
        i = ctx + torch.arange(n, device=DEV)[:, None]
        key = torch.arange(L, device=DEV)
        seen = (key <= i) | (key < prefix)
        if c["window"]:
            seen &= i - key < c["window"]
        for d in cuts[1:] if c["documents"] else ():
            seen &= ~((key < d) & (i >= d))
        o = torch.empty(n, hq, D, device=DEV, dtype=torch.float64)
        lse = torch.empty(n, hq, device=DEV, dtype=torch.float64)
        for h in range(hq):
            s = q[:, h] @ k[:, h // (hq // hkv)].T / math.sqrt(D)
            if c["cap"]:
                s = c["cap"] * torch.tanh(s / c["cap"])
            if c["slopes"]:
                s = s - st["slopes"][h].double() * (i - key).abs()
            s = torch.where(seen, s, -math.inf)
            lse[:, h] = torch.logsumexp(s, -1)
            p = torch.where(seen, torch.exp(s - lse[:, h, None]), 0.0)
            o[:, h] = p @ v[:, h // (hq // hkv)]
        outs.append(o)
        lses.append(lse)
    return [torch.cat(outs), torch.cat(lses)]


def _exact_drafts(st):
    c = st["case"]
    K, V = c["drafts"], c["vocab"]
    tokens, accepted, kept = [], [], []
    for b, n in enumerate(st["draft_lens"].tolist()):
        drafts, u = st["drafts"][b].tolist(), st["u"][b].double().tolist()
        j = 0
        while j < n:
            qx = 1.0 if st["q"] is None else float(st["q"][b, j, drafts[j]])
            if not u[j] * qx < float(st["p"][b, j, drafts[j]]):
                break
            j += 1
        w = st["p"][b, j].double()
        if j < n:
            if st["q"] is None:
                less = w.clone()
                less[drafts[j]] = 0.0
            else:
                less = torch.relu(w - st["q"][b, j].double())
            w = less if float(less.sum()) > 0 else w
        cum = torch.cumsum(w, 0)
        token = int(torch.searchsorted(cum, u[K] * float(cum[-1]), right=True))
        tokens.append(drafts[:j] + [min(token, V - 1)] + [-1] * (K - j))
        accepted.append(j)
        kept.append(int(st["seq_lens"][b]) - (n - j))
    return [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (tokens, accepted, kept)]


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "drafts": _exact_drafts}.get(case["op"],
                                                                  _exact_attention)(st)
