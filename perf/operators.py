"""Attention with grouped heads over packed prompts, the 8-bit paged cache that serving keeps of its keys and
values, and the attention of new tokens over that cache: the cases that are measured, the operators' plain forms
and their definitions in 64 bits.

A case's "op" is one of
  prefill  O and LSE of packed prompts, causal, H query heads over Hk key/value heads
  train    the same forward and its backward: O, dQ, dK, dV
  store    keys and values of new tokens into the paged cache: e4m3 codes with one power-of-two scale for each
           block of tokens and head
  decode   Nq new tokens of each sequence against the cache
"""
import math

import torch

own = False

E4M3_MAX = 448.0
SCALE_FLOOR = -64  # exponent of the smallest scale


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one short prompt of a small model: latency
        dict(name="prefill_short", op="prefill", nseq=1, lo=100, hi=100, pad=0, H=4, Hk=1, d=64),
        # a serving batch of prompts of mixed lengths
        dict(name="prefill_mixed", op="prefill", nseq=16, lo=64, hi=2048, pad=0, H=32, Hk=8, d=128),
        # one long document
        dict(name="prefill_long", op="prefill", nseq=1, lo=8192, hi=8192, pad=0, H=32, Hk=8, d=128),
        # a few short samples, one of them a single token
        dict(name="train_short", op="train", nseq=3, lo=1, hi=300, pad=0, H=8, Hk=2, d=64),
        # a packed training batch that does not fill its buffer
        dict(name="train_mixed", op="train", nseq=8, lo=64, hi=2048, pad=77, H=32, Hk=8, d=128),
        # two long samples, one key/value head for eight query heads
        dict(name="train_long", op="train", nseq=2, lo=3900, hi=4100, pad=0, H=32, Hk=4, d=64),
        # one decoding step's tokens of a batch
        dict(name="store_step", op="store", B=64, lo=1, hi=1, start=2000, Hk=8, d=128, block=64),
        # the prompts of a batch, some of them behind a cached beginning
        dict(name="store_prompt", op="store", B=16, lo=64, hi=4096, start=40, Hk=8, d=128, block=16),
        # a single conversation: latency
        dict(name="decode_one", op="decode", B=1, lo=777, hi=777, Nq=1, H=32, Hk=8, d=128, block=16),
        # a serving batch of ragged lengths
        dict(name="decode_batch", op="decode", B=64, lo=100, hi=8192, Nq=1, H=32, Hk=8, d=128, block=64),
        # long contexts, every head with keys and values of its own
        dict(name="decode_long", op="decode", B=4, lo=32768, hi=32768, Nq=1, H=32, Hk=32, d=128, block=128),
        # four tokens at once of each sequence, as when drafted tokens are verified
        dict(name="decode_draft", op="decode", B=16, lo=500, hi=4096, Nq=4, H=64, Hk=8, d=64, block=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "train", "store", "decode"])
    d = rng.choice([64, 128])
    if op in ("prefill", "train"):
        Hk, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8])
        H = Hk * G
        nseq = _log(rng, 1, 24)
        # padded scores of at most 2^29 values, and no more work than the long prompt's
        hi = _log(rng, 1, max(2, min(8000, int(math.sqrt(2.0 ** 29 / (nseq * H))))))
        lo = rng.randint(1, hi)
        return dict(op=op, nseq=nseq, lo=lo, hi=hi, pad=rng.choice([0, 0, 1, 130]), H=H, Hk=Hk, d=d)
    Hk, block = rng.choice([1, 2, 5, 8]), rng.choice([16, 32, 64, 128])
    if op == "store":
        B, hi = _log(rng, 1, 48), _log(rng, 1, 2000)
        return dict(op=op, B=B, lo=rng.randint(1, hi), hi=hi, start=rng.choice([0, 1, 17, 1000]), Hk=Hk, d=d, block=block)
    B = _log(rng, 1, 48)
    hi = _log(rng, 8, 8000)
    return dict(op=op, B=B, lo=rng.randint(8, hi), hi=hi, Nq=rng.choice([1, 1, 2, 5, 8]), H=Hk * rng.choice([1, 2, 4, 7, 8]), Hk=Hk, d=d,
                block=block)


def _lengths(n, lo, hi):
    """n lengths spread over [lo, hi], the last of them hi."""
    return [lo + int((hi - lo) * ((0.6180339887498949 * (i + 1)) % 1.0)) for i in range(n - 1)] + [hi]


def _starts(case):
    """Cached tokens of each sequence before the store: up to `start`, some sequences without any."""
    return [(case["start"] * (7 * i + 3)) // 11 % (case["start"] + 1) if i % 5 else 0 for i in range(case["B"])]


# ------------------------------------------------------------------------------------------------ inputs
def _gains(g, d, spread):
    return torch.exp(spread * torch.randn(d, generator=g, device="cuda"))


def _pow2(amax):
    """The smallest power of two s with amax <= 448 s, not below 2^SCALE_FLOOR (amax: fp32). Made of its exponent's bits:
    a power function need not be exact."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=SCALE_FLOOR)
    return ((torch.where(amax > 0, e, SCALE_FLOOR).int() + 127) << 23).view(torch.float32)


def _cache(g, pages, Hk, block, d, spread):
    """A pool of filled pages: codes and scales of normal values with uneven channels."""
    x = torch.randn(pages, Hk, block, d, generator=g, device="cuda") * _gains(g, d, spread)
    s = _pow2(x.abs().amax((2, 3)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d, Hk = case["d"], case["Hk"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    i32 = dict(dtype=torch.int32, device="cuda")
    if case["op"] in ("prefill", "train"):
        lens = _lengths(case["nseq"], case["lo"], case["hi"])
        T, H = sum(lens) + case["pad"], case["H"]
        gains = _gains(g, d, 0.3)
        st = dict(case=case, max_seqlen=max(lens), cu=torch.tensor([0] + lens, **i32).cumsum(0, dtype=torch.int32),
                  q=normal(T, H, d).bfloat16(), k=(normal(T, Hk, d) * gains).bfloat16(), v=normal(T, Hk, d).bfloat16())
        if case["op"] == "train":
            st["do"] = normal(T, H, d).bfloat16()
            for n in "qkv":
                st[n].requires_grad_()
        return st
    B, block = case["B"], case["block"]
    lens = _lengths(B, case["lo"], case["hi"])
    starts = _starts(case) if case["op"] == "store" else [0] * B
    cols = max(-(-(a + n) // block) for a, n in zip(starts, lens))
    pages = sum(-(-(a + n) // block) for a, n in zip(starts, lens)) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table, at = torch.zeros(B, cols, **i32), 0
    for b in range(B):  # each sequence's pages lie anywhere in the pool
        n = -(-(starts[b] + lens[b]) // block)
        table[b, :n] = order[at:at + n]
        at += n
    ck, sk = _cache(g, pages, Hk, block, d, 0.5)
    cv, sv = _cache(g, pages, Hk, block, d, 0.2)
    st = dict(case=case, table=table, ck=ck, cv=cv, sk=sk, sv=sv)
    if case["op"] == "store":
        T = sum(lens)
        st |= dict(k=(normal(T, Hk, d) * _gains(g, d, 0.5)).bfloat16(), v=(normal(T, Hk, d) * _gains(g, d, 0.2)).bfloat16(),
                   cu=torch.tensor([0] + lens, **i32).cumsum(0, dtype=torch.int32), start=torch.tensor(starts, **i32),
                   max_new=max(lens))
    else:
        st |= dict(q=normal(B, case["Nq"], case["H"], d).bfloat16(), lens=torch.tensor(lens, **i32), max_seqlen=max(lens))
    return st


# ------------------------------------------------------------------------------------------------ the pass
def run(state):
    return {"prefill": _prefill, "train": _train, "store": _store, "decode": _decode}[state["case"]["op"]](state)


def _padded(st):
    """(rows [nseq, M], which of them exist, key visible to query [M, M] and within the sequence)."""
    cu = st["cu"].long()
    at = torch.arange(st["max_seqlen"], device=cu.device)
    live = at < (cu[1:] - cu[:-1])[:, None]
    rows = torch.where(live, cu[:-1, None] + at, 0)
    seen = (at[None, :] <= at[:, None])[None] & live[:, None, :]
    return rows, live, seen


def _group(x, rows, Hk):
    """[T, Hk·G, d] -> fp32 [nseq, Hk, G, M, d]"""
    n, M = rows.shape
    return x[rows].float().reshape(n, M, Hk, -1, x.shape[2]).permute(0, 2, 3, 1, 4)


def _ungroup(x, rows, live, T):
    """[nseq, Hk, G, M, d] -> [T, Hk·G, d], zeros in rows behind the last sequence"""
    n, Hk, G, M, d = x.shape
    out = torch.zeros(T, Hk * G, d, device=x.device)
    out[rows[live]] = x.permute(0, 3, 1, 2, 4).reshape(n, M, Hk * G, d)[live]
    return out


def _softmax_parts(s, seen):
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m)
    return m, p, p.sum(-1, keepdim=True)


def _prefill(st):
    if own:
        import io_aware_attention_flash_gb300 as fa

        return fa.attention_forward_grouped(st["q"], st["k"], st["v"], st["cu"], st["max_seqlen"], causal=True)
    Hk, d, T = st["k"].shape[1], st["q"].shape[2], st["q"].shape[0]
    rows, live, seen = _padded(st)
    q, k, v = (_group(st[n], rows, Hk) for n in "qkv")
    m, p, l = _softmax_parts(q @ k.transpose(-1, -2) * d ** -0.5, seen)
    lse = torch.full((q.shape[1] * q.shape[2], T), -math.inf, device=q.device)
    lse[:, rows[live]] = (m + torch.log(l)).flatten(1, 2)[..., 0].permute(0, 2, 1)[live].T
    return _ungroup(p @ v / l, rows, live, T).bfloat16(), lse


def _train(st):
    if own:
        import io_aware_attention_flash_gb300 as fa

        o = fa.flash_attention_grouped(st["q"], st["k"], st["v"], st["cu"], st["max_seqlen"], causal=True)
        return (o, *torch.autograd.grad(o, (st["q"], st["k"], st["v"]), st["do"]))
    with torch.no_grad():
        Hk, d, T = st["k"].shape[1], st["q"].shape[2], st["q"].shape[0]
        rows, live, seen = _padded(st)
        q, k, v = (_group(st[n], rows, Hk) for n in "qkv")
        do = _group(st["do"], rows, Hk) * live[:, None, None, :, None]
        _, p, l = _softmax_parts(q @ k.transpose(-1, -2) * d ** -0.5, seen)
        p = p / l
        o = p @ v
        dv = (p.transpose(-1, -2) @ do).sum(2, keepdim=True)
        dp = do @ v.transpose(-1, -2)
        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * d ** -0.5
        dq, dk = ds @ k, (ds.transpose(-1, -2) @ q).sum(2, keepdim=True)
        return tuple(_ungroup(x, rows, live, T).bfloat16() for x in (o, dq, dk, dv))


def _quantise(new, codes, scale, cu, start, table, max_new):
    """The tokens of `new` [T, Hk, d] into codes [pages, Hk, block, d] and scale [pages, Hk], in place."""
    block, cols = codes.shape[2], table.shape[1]
    cu, start = cu.long(), start.long()
    count = cu[1:] - cu[:-1]
    blk = start[:, None] // block + torch.arange(-(-max_new // block) + 1, device=cu.device)  # [B, NB]
    pos = blk[..., None] * block + torch.arange(block, device=cu.device)  # [B, NB, block]
    is_new = (pos >= start[:, None, None]) & (pos < (start + count)[:, None, None])
    touched = is_new.any(-1)
    is_old = (pos < start[:, None, None])[touched]
    is_new, pos = is_new[touched], pos[touched]
    seq = torch.arange(cu.numel() - 1, device=cu.device)[:, None].expand_as(touched)[touched]
    page = table.long()[seq, blk[touched].clamp(max=cols - 1)]
    src = torch.where(is_new, cu[seq][:, None] + pos - start[seq][:, None], 0)
    x = new[src].float().masked_fill(~is_new[..., None, None], 0.0)  # [n, block, Hk, d]
    s = _pow2(x.abs().amax((1, 3)))  # [n, Hk]
    before = scale[page]
    s = torch.where(is_old.any(1, keepdim=True), torch.maximum(s, before), s)
    held = codes[page].float().permute(0, 2, 1, 3) * before[:, None, :, None]
    x = torch.where(is_old[..., None, None], held, x) / s[:, None, :, None]
    x = x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    n, slot = (is_old | is_new).nonzero(as_tuple=True)
    codes.view(torch.uint8)[page[n], :, slot] = x[n, slot]
    scale[page] = s


def _store(st):
    args = st["table"], st["cu"], st["start"], st["max_new"]
    if own:
        import io_aware_attention_flash_gb300 as fa

        fa.cache8_store(st["k"], st["v"], fa.Cache8(st["ck"], st["cv"], st["sk"], st["sv"]), *args)
    else:
        table, cu, start, max_new = args
        _quantise(st["k"], st["ck"], st["sk"], cu, start, table, max_new)
        _quantise(st["v"], st["cv"], st["sv"], cu, start, table, max_new)
    return st["ck"], st["cv"], st["sk"], st["sv"]


def _decode(st):
    if own:
        import io_aware_attention_flash_gb300 as fa

        return fa.attention_decode_cache8(st["q"], fa.Cache8(st["ck"], st["cv"], st["sk"], st["sv"]), st["table"], st["lens"],
                                          st["max_seqlen"], causal=True)
    B, Nq, H, d = st["q"].shape
    Hk, block = st["ck"].shape[1:3]
    table, lens = st["table"].long(), st["lens"].long()
    at = torch.arange(table.shape[1] * block, device=lens.device)

    def values(codes, scale):  # -> [B, Hk, L, d]; slots past the length hold anything
        x = (codes[table].float() * scale[table][..., None, None]).transpose(1, 2).flatten(2, 3)
        return x.masked_fill((at >= lens[:, None])[:, None, :, None], 0.0)

    q = st["q"].float().reshape(B, Nq, Hk, H // Hk, d).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hk, G·Nq, d]
    last = (lens[:, None] - Nq + torch.arange(Nq, device=lens.device)).repeat(1, H // Hk)  # [B, G·Nq]
    s = q @ values(st["ck"], st["sk"]).transpose(-1, -2) * d ** -0.5
    s = s.masked_fill((at > last[..., None])[:, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    o = p @ values(st["cv"], st["sv"]) / l.clamp(min=1e-30)
    o = o.reshape(B, Hk, H // Hk, Nq, d).permute(0, 3, 1, 2, 4).reshape(B, Nq, H, d)
    return o.bfloat16(), (m + torch.log(l)).reshape(B, H, Nq)


# ------------------------------------------------------------------------------------------------ what it cannot do without
def work(case):
    d, Hk = case["d"], case["Hk"]
    if case["op"] in ("prefill", "train"):
        lens = _lengths(case["nseq"], case["lo"], case["hi"])
        H, rows = case["H"], sum(lens)
        flops = 4.0 * d * H * sum(n * (n + 1) / 2 for n in lens)
        if case["op"] == "prefill":
            return {"bytes": rows * (2 * 2 * H * d + 2 * 2 * Hk * d + 4 * H), "flops": flops}
        return {"bytes": rows * (4 * 2 * H * d + 4 * 2 * Hk * d), "flops": 3.5 * flops}
    lens = _lengths(case["B"], case["lo"], case["hi"])
    if case["op"] == "store":
        new = sum(lens) * Hk * d * 2
        return {"bytes": new * 3, "flops": 4.0 * new}
    rows = case["B"] * case["Nq"] * case["H"]
    return {"bytes": sum(lens) * Hk * d * 2 + rows * (4 * d + 4), "flops": 4.0 * d * case["H"] * case["Nq"] * sum(lens)}


# ------------------------------------------------------------------------------------------------ the definitions, in 64 bits
def _attend64(q, k, v, first):
    """softmax(q kᵀ / sqrt(d)) row by row in 64 bits: row i sees keys 0 .. first + i. -> P, O, LSE"""
    n, m = q.shape[0], k.shape[0]
    s = (q @ k.T) / math.sqrt(q.shape[1])
    hidden = torch.arange(m, device=q.device)[None] > first + torch.arange(n, device=q.device)[:, None]
    s[hidden] = -math.inf
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - lse[:, None])
    p[hidden] = 0.0
    return p, p @ v, lse


def _exp2_64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """x (64 bits) to the nearest e4m3 value, ties to even: 4 significant bits down to 2^-6, steps of 2^-9 below."""
    step = _exp2_64((torch.frexp(x)[1] - 4).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    with torch.no_grad():
        st = prepare(case, seed)
        Hk, d = case["Hk"], case["d"]
        if case["op"] in ("prefill", "train"):
            H, T = case["H"], st["q"].shape[0]
            G, cu = H // Hk, st["cu"].tolist()
            q, k, v = (st[n].double() for n in "qkv")
            o, dq, lse = torch.zeros_like(q), torch.zeros_like(q), torch.full((H, T), -math.inf, dtype=torch.float64, device="cuda")
            dk, dv = torch.zeros_like(k), torch.zeros_like(v)
            for a, b in zip(cu[:-1], cu[1:]):
                for h in range(H):
                    kh, vh = k[a:b, h // G], v[a:b, h // G]
                    p, o[a:b, h], lse[h, a:b] = _attend64(q[a:b, h], kh, vh, 0)
                    if case["op"] == "train":
                        do = st["do"][a:b, h].double()
                        dv[a:b, h // G] += p.T @ do
                        dp = do @ vh.T
                        ds = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(d)
                        dq[a:b, h] = ds @ kh
                        dk[a:b, h // G] += ds.T @ q[a:b, h]
            return (o, lse) if case["op"] == "prefill" else (o, dq, dk, dv)
        table, block = st["table"].tolist(), case["block"]
        if case["op"] == "decode":
            o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
            B, Nq, H, _ = o.shape
            lse = torch.full((B, H, Nq), -math.inf, dtype=torch.float64, device="cuda")
            G = H // Hk
            for b, n in enumerate(st["lens"].tolist()):
                pages = table[b][:-(-n // block)]
                k, v = ((c[pages].double() * s[pages].double()[..., None, None]).transpose(0, 1).flatten(1, 2)[:, :n]
                        for c, s in ((st["ck"], st["sk"]), (st["cv"], st["sv"])))
                for h in range(H):
                    seen = slice(max(0, Nq - n), Nq)  # the first new tokens of a cache shorter than Nq see nothing
                    _, o[b, seen, h], lse[b, h, seen] = _attend64(st["q"][b, seen, h].double(), k[h // G], v[h // G],
                                                                  max(0, n - Nq))
            return o, lse
        out = []
        cu, start = st["cu"].tolist(), st["start"].tolist()
        for x, codes, scale in ((st["k"], st["ck"], st["sk"]), (st["v"], st["cv"], st["sv"])):
            codes, scale, x = codes.double(), scale.double(), x.double()
            for b in range(case["B"]):
                end, page_of = start[b] + cu[b + 1] - cu[b], table[b]
                for j in range(start[b] // block, -(-end // block)):
                    lo, hi = max(start[b], j * block), min(end, (j + 1) * block)
                    page, old = page_of[j], max(0, start[b] - j * block)
                    new = x[cu[b] + lo - start[b]:cu[b] + hi - start[b]].transpose(0, 1)  # [Hk, n, d]
                    half, e = torch.frexp(new.abs().amax((1, 2)) / E4M3_MAX)  # an exact power of two has the fraction 1/2
                    s = _exp2_64((e - (half <= 0.5).int()).clamp(min=SCALE_FLOOR))
                    if old:
                        s = torch.maximum(s, scale[page])
                        codes[page, :, :old] = _round_e4m3(codes[page, :, :old] * (scale[page] / s)[:, None, None])
                    codes[page, :, lo - j * block:hi - j * block] = _round_e4m3(new / s[:, None, None])
                    scale[page] = s
            out += [codes, scale]
        return out[0], out[2], out[1], out[3]
