"""Rotary positions for training, the append of rotated keys and of values to the 8-bit paged cache, and the attention
of a chunk of new tokens over that cache: the cases that are measured, the operators' plain forms and their definitions
in 64 bits.

A case's "op" is one of
  rotate  queries and keys of a packed batch turned by their tokens' positions (one axis, or time, height and width),
          and the gradients turned back: q', k', dq, dk
  append  one step's or one prompt's tokens: queries turned, keys turned and stored with the values as e4m3 codes with
          one power-of-two scale for each page and head: q', codes and scales
  chunk   the new tokens of each sequence (a prompt's next piece, a single token) against the cache that already holds
          them: O and LSE
"""
import math

import torch

own = False

E4M3_MAX = 448.0
SCALE_FLOOR = -64  # exponent of the smallest scale
BASE = 10000.0


# ------------------------------------------------------------------------------------------------ cases
# pairs: rotated pairs of a head's dimensions (the rest passes unturned); axes: position axes, shared out over the pairs;
# interleaved: a pair is two neighbours (else one dimension of each half); far: first position
def listed():
    return [
        # one short sample of a small model: latency
        dict(name="rotate_short", op="rotate", T=100, H=4, Hk=1, d=64, pairs=32, axes=1, interleaved=False, far=0),
        # a packed training batch of text
        dict(name="rotate_text", op="rotate", T=16421, H=32, Hk=8, d=128, pairs=64, axes=1, interleaved=False, far=0),
        # frames of a video, of which a long part came before: positions in time, height and width, neighbours paired
        dict(name="rotate_video", op="rotate", T=9000, H=16, Hk=16, d=128, pairs=48, axes=3, interleaved=True, far=1000000),
        # one decoding step's tokens of a batch
        dict(name="append_step", op="append", B=64, lo=1, hi=1, start=2000, H=32, Hk=8, d=128, block=64, pairs=64, axes=1,
             interleaved=False),
        # the prompts of a batch, some of them behind a cached beginning
        dict(name="append_prompt", op="append", B=16, lo=64, hi=4096, start=40, H=32, Hk=8, d=128, block=16, pairs=64, axes=1,
             interleaved=False),
        # a few images with their text
        dict(name="append_image", op="append", B=3, lo=577, hi=2000, start=17, H=8, Hk=2, d=64, block=32, pairs=32, axes=3,
             interleaved=False),
        # a short question behind a cached beginning: latency
        dict(name="chunk_short", op="chunk", B=1, nlo=37, nhi=37, lo=777, hi=777, H=4, Hk=1, d=64, block=16, causal=True),
        # a serving step: single tokens of some sequences, pieces of prompts of others
        dict(name="chunk_mixed", op="chunk", B=16, nlo=1, nhi=512, lo=100, hi=8192, H=32, Hk=8, d=128, block=64, causal=True),
        # the last piece of a long document
        dict(name="chunk_document", op="chunk", B=1, nlo=2048, nhi=2048, lo=32768, hi=32768, H=32, Hk=8, d=128, block=128,
             causal=True),
        # a few tokens at the end of long contexts
        dict(name="chunk_few", op="chunk", B=4, nlo=12, nhi=12, lo=32768, hi=32768, H=32, Hk=8, d=128, block=16, causal=True),
        # pieces of prompts of a smaller model
        dict(name="chunk_small_heads", op="chunk", B=6, nlo=100, nhi=700, lo=700, hi=4096, H=64, Hk=8, d=64, block=32, causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "append", "chunk", "chunk"])
    d, Hk = rng.choice([64, 128]), rng.choice([1, 2, 3, 5, 8])
    H = Hk * rng.choice([1, 2, 3, 4, 7, 8])
    turn = dict(pairs=rng.choice([d // 2, d // 2, d // 4, d // 2 - 8]), axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.4)
    if op == "rotate":
        # no more elements than the packed batch of text
        return dict(op=op, T=_log(rng, 1, 80000000 // ((H + Hk) * d)), H=H, Hk=Hk, d=d, far=rng.choice([0, 0, 5000, 20000000]), **turn)
    block = rng.choice([16, 32, 64, 128])
    if op == "append":
        B = _log(rng, 1, 48)
        hi = _log(rng, 1, max(2, min(1500, 160000000 // (B * (H + 2 * Hk) * d))))
        return dict(op=op, B=B, lo=rng.randint(1, hi), hi=hi, start=rng.choice([0, 1, 17, 1000]), H=H, Hk=Hk, d=d, block=block, **turn)
    B, hi = _log(rng, 1, 24), _log(rng, 16, 20000)
    # scores of one sequence of at most 2^29 values, and no more work than the long document's
    nhi = _log(rng, 1, max(2, min(hi, 3000, 2 ** 29 // (hi * H), 2 ** 31 // (hi * H * B))))
    return dict(op=op, B=B, nlo=rng.randint(1, nhi), nhi=nhi, lo=rng.randint(nhi, hi), hi=hi, H=H, Hk=Hk, d=d, block=block,
                causal=rng.random() < 0.85)


def _lengths(n, lo, hi):
    """n lengths spread over [lo, hi], the last of them hi."""
    return [lo + int((hi - lo) * ((0.6180339887498949 * (i + 1)) % 1.0)) for i in range(n - 1)] + [hi]


def _chunks(case):
    """(new tokens, cached tokens with the new ones) of each sequence; every third sequence has the fewest new ones."""
    new = [case["nlo"] if i % 3 == 1 else n for i, n in enumerate(_lengths(case["B"], case["nlo"], case["nhi"]))]
    return new, [max(n, L) for n, L in zip(new, _lengths(case["B"], case["lo"], case["hi"])[::-1])]


def _starts(case):
    """Cached tokens of each sequence before the append: up to `start`, some sequences without any."""
    return [(case["start"] * (7 * i + 3)) // 11 % (case["start"] + 1) if i % 5 else 0 for i in range(case["B"])]


def _grid(n, first):
    """Time, height and width of n patches, 24 wide and 18 high a frame."""
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    return torch.stack([first + at // (24 * 18), at // 24 % 18, at % 24])


def _axis_of(case):
    """The axis of each pair: runs of pairs, the first a little longer."""
    m, n = case["pairs"], case["axes"]
    return [min(i * n // (m + n - 1), n - 1) for i in range(m)] if n > 1 else [0] * m


def _inv_freq(case):
    return [BASE ** (-i / case["pairs"]) for i in range(case["pairs"])]


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


def _plan(st, case):
    """What a program keeps of its rotary frequencies."""
    if own:
        import io_aware_attention_flash_gb300 as fa

        st["rotary"] = fa.rotary_plan(_inv_freq(case), axis=_axis_of(case), interleaved=case["interleaved"])
    else:
        st["inv_freq"] = torch.tensor(_inv_freq(case), dtype=torch.float64, device="cuda")
        st["axis"] = torch.tensor(_axis_of(case), device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d, H, Hk = case["d"], case["H"], case["Hk"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    i32 = dict(dtype=torch.int32, device="cuda")
    if case["op"] == "rotate":
        T = case["T"]
        st = dict(case=case, q=normal(T, H, d).bfloat16().requires_grad_(), k=(normal(T, Hk, d) * _gains(g, d, 0.4)).bfloat16().requires_grad_(),
                  dq=normal(T, H, d).bfloat16(), dk=normal(T, Hk, d).bfloat16())
        if case["axes"] > 1:
            st["positions"] = _grid(T, case["far"])[:case["axes"]].contiguous()
        else:  # samples of 1 to 4000 tokens, the position counted from each one's beginning
            at = torch.arange(T, **i32)
            cut = torch.randint(1, 4000, (T // 1000 + 1,), generator=g, device="cuda").cumsum(0)
            first = torch.cat([cut.new_zeros(1), cut])[torch.searchsorted(cut, at, right=True)]
            st["positions"] = (at - first + case["far"]).int()
        _plan(st, case)
        return st
    B, block = case["B"], case["block"]
    if case["op"] == "append":
        new, before = _lengths(B, case["lo"], case["hi"]), _starts(case)
        lens = [a + n for a, n in zip(before, new)]
    else:
        new, lens = _chunks(case)
    cols = max(-(-n // block) for n in lens)
    pages = sum(-(-n // block) for n in lens) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table, at = torch.zeros(B, cols, **i32), 0
    for b in range(B):  # each sequence's pages lie anywhere in the pool
        n = -(-lens[b] // block)
        table[b, :n] = order[at:at + n]
        at += n
    ck, sk = _cache(g, pages, Hk, block, d, 0.5)
    cv, sv = _cache(g, pages, Hk, block, d, 0.2)
    T = sum(new)
    st = dict(case=case, table=table, ck=ck, cv=cv, sk=sk, sv=sv, q=normal(T, H, d).bfloat16(), max_new=max(new),
              cu=torch.tensor([0] + new, **i32).cumsum(0, dtype=torch.int32))
    if case["op"] == "append":
        st |= dict(k=(normal(T, Hk, d) * _gains(g, d, 0.5)).bfloat16(), v=(normal(T, Hk, d) * _gains(g, d, 0.2)).bfloat16(),
                   start=torch.tensor(before, **i32), positions=None)
        if case["axes"] > 1:
            st["positions"] = torch.cat([_grid(n, a) for n, a in zip(new, before)], 1)[:case["axes"]].contiguous()
        _plan(st, case)
    else:
        st |= dict(lens=torch.tensor(lens, **i32), max_seqlen=max(lens), new=new, held=lens)
    return st


# ------------------------------------------------------------------------------------------------ the pass
def run(state):
    return {"rotate": _rotate, "append": _append, "chunk": _chunk}[state["case"]["op"]](state)


def _cos_sin(st, positions):
    """Cosine and sine of each token's angles (formed in 64 bits), fp32 [T, 1, pairs]."""
    at = positions.double().reshape(-1, positions.shape[-1])[st["axis"]]  # [pairs, T]
    angle = (at.T * st["inv_freq"])[:, None]
    return torch.cos(angle).float(), torch.sin(angle).float()


def _turn(x, cos, sin, interleaved):
    """x [T, heads, d] in 32 bits with its first 2 · pairs dimensions turned."""
    m = cos.shape[-1]
    x = x.float()
    if interleaved:
        a, b = x[..., 0:2 * m:2], x[..., 1:2 * m:2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :m], x[..., m:2 * m]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([head, x[..., 2 * m:]], -1)


def _rotate(st):
    if own:
        import io_aware_attention_flash_gb300 as fa

        q, k = fa.rotary_embedding(st["q"], st["k"], st["positions"], st["rotary"])
        return (q, k, *torch.autograd.grad((q, k), (st["q"], st["k"]), (st["dq"], st["dk"])))
    with torch.no_grad():
        cos, sin = _cos_sin(st, st["positions"])
        il = st["case"]["interleaved"]
        return tuple(_turn(st[n], cos, s, il).bfloat16() for n, s in (("q", sin), ("k", sin), ("dq", -sin), ("dk", -sin)))


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


def _append(st):
    if own:
        import io_aware_attention_flash_gb300 as fa

        q = fa.cache8_store_rotary(st["q"], st["k"], st["v"], fa.Cache8(st["ck"], st["cv"], st["sk"], st["sv"]), st["table"], st["cu"],
                                   st["start"], st["max_new"], st["rotary"], st["positions"])
        return q, st["ck"], st["cv"], st["sk"], st["sv"]
    cu, start, positions = st["cu"], st["start"], st["positions"]
    if positions is None:  # a token's place in its sequence
        row = torch.arange(st["q"].shape[0], device=cu.device)
        b = torch.searchsorted(cu[1:].long(), row, right=True)
        positions = start[b] + row - cu[b]
    cos, sin = _cos_sin(st, positions)
    il = st["case"]["interleaved"]
    _quantise(_turn(st["k"], cos, sin, il), st["ck"], st["sk"], cu, start, st["table"], st["max_new"])
    _quantise(st["v"], st["cv"], st["sv"], cu, start, st["table"], st["max_new"])
    return _turn(st["q"], cos, sin, il).bfloat16(), st["ck"], st["cv"], st["sk"], st["sv"]


def _chunk(st):
    causal = st["case"]["causal"]
    if own:
        import io_aware_attention_flash_gb300 as fa

        return fa.attention_chunk_cache8(st["q"], fa.Cache8(st["ck"], st["cv"], st["sk"], st["sv"]), st["table"], st["cu"], st["lens"],
                                         st["max_new"], st["max_seqlen"], causal=causal)
    T, H, d = st["q"].shape
    Hk, block = st["ck"].shape[1:3]
    G = H // Hk
    o = torch.empty(T, H, d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(H, T, device="cuda")
    first = 0
    for b, (n, L) in enumerate(zip(st["new"], st["held"])):
        pages = st["table"][b, :-(-L // block)].long()
        k, v = ((c[pages].float() * s[pages][..., None, None]).transpose(0, 1).flatten(1, 2)[:, :L]
                for c, s in ((st["ck"], st["sk"]), (st["cv"], st["sv"])))  # [Hk, L, d]
        q = st["q"][first:first + n].float().reshape(n, Hk, G, d).permute(1, 2, 0, 3).flatten(1, 2)  # [Hk, G·n, d]
        s = q @ k.transpose(1, 2) * d ** -0.5
        if causal:
            at = torch.arange(L, device="cuda")
            s.view(Hk, G, n, L).masked_fill_(at > (L - n + torch.arange(n, device="cuda"))[:, None], -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        l = p.sum(-1, keepdim=True)
        o[first:first + n] = (p @ v / l).reshape(Hk, G, n, d).permute(2, 0, 1, 3).reshape(n, H, d)
        lse[:, first:first + n] = (m + torch.log(l)).reshape(H, n)
        first += n
    return o, lse


# ------------------------------------------------------------------------------------------------ what it cannot do without
def work(case):
    d, H, Hk = case["d"], case["H"], case["Hk"]
    turned = 2 * case.get("pairs", 0)
    if case["op"] == "rotate":
        rows = case["T"] * (H + Hk)
        return {"bytes": rows * d * 2 * 4 + 4 * case["axes"] * case["T"], "flops": 2 * 3.0 * rows * turned}
    if case["op"] == "append":
        rows = sum(_lengths(case["B"], case["lo"], case["hi"]))
        return {"bytes": rows * d * (2 * 3 * Hk + 4 * H), "flops": rows * (3.0 * (H + Hk) * turned + 4.0 * Hk * d)}
    new, lens = _chunks(case)
    if case["causal"]:
        pairs = sum(n * (L - n) + n * (n + 1) / 2 for n, L in zip(new, lens))
    else:
        pairs = sum(n * L for n, L in zip(new, lens))
    return {"bytes": sum(lens) * Hk * d * 2 + sum(new) * H * (4 * d + 4), "flops": 4.0 * d * H * pairs}


# ------------------------------------------------------------------------------------------------ the definitions, in 64 bits
def _exp2_64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """x (64 bits) to the nearest e4m3 value, ties to even: 4 significant bits down to 2^-6, steps of 2^-9 below."""
    step = _exp2_64((torch.frexp(x)[1] - 4).clamp(min=-9))
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _turn64(x, positions, case, back=False):
    """Each pair as a complex number, times e^(i angle)."""
    m, x = case["pairs"], x.detach().double()
    angle = torch.stack([positions.reshape(-1, x.shape[0])[a].double() * f for a, f in zip(_axis_of(case), _inv_freq(case))], 1)
    unit = torch.polar(torch.ones_like(angle), -angle if back else angle)[:, None]
    out = x.clone()
    if case["interleaved"]:
        out[..., :2 * m] = torch.view_as_real(torch.view_as_complex(x[..., :2 * m].reshape(*x.shape[:2], m, 2).contiguous()) * unit).flatten(-2)
    else:
        z = torch.complex(x[..., :m].contiguous(), x[..., m:2 * m].contiguous()) * unit
        out[..., :m], out[..., m:2 * m] = z.real, z.imag
    return out


def exact(case, seed):
    with torch.no_grad():
        st = prepare(case, seed)
        Hk, d, H = case["Hk"], case["d"], case["H"]
        if case["op"] == "rotate":
            p = st["positions"]
            return tuple(_turn64(st[n], p, case, back) for n, back in (("q", False), ("k", False), ("dq", True), ("dk", True)))
        table, block, cu = st["table"].tolist(), case["block"], st["cu"].tolist()
        if case["op"] == "append":
            start = st["start"].tolist()
            p = st["positions"]
            if p is None:
                p = torch.cat([torch.arange(a, a + e - s, device="cuda") for a, s, e in zip(start, cu[:-1], cu[1:])])
            out = []
            for x, codes, scale in ((_turn64(st["k"], p, case), st["ck"], st["sk"]), (st["v"].double(), st["cv"], st["sv"])):
                codes, scale = codes.double(), scale.double()
                for b in range(case["B"]):
                    end = start[b] + cu[b + 1] - cu[b]
                    for j in range(start[b] // block, -(-end // block)):
                        lo, hi = max(start[b], j * block), min(end, (j + 1) * block)
                        page, old = table[b][j], max(0, start[b] - j * block)
                        new = x[cu[b] + lo - start[b]:cu[b] + hi - start[b]].transpose(0, 1)  # [Hk, n, d]
                        half, e = torch.frexp(new.abs().amax((1, 2)) / E4M3_MAX)  # an exact power of two has the fraction 1/2
                        s = _exp2_64((e - (half <= 0.5).int()).clamp(min=SCALE_FLOOR))
                        if old:
                            s = torch.maximum(s, scale[page])
                            codes[page, :, :old] = _round_e4m3(codes[page, :, :old] * (scale[page] / s)[:, None, None])
                        codes[page, :, lo - j * block:hi - j * block] = _round_e4m3(new / s[:, None, None])
                        scale[page] = s
                out += [codes, scale]
            return _turn64(st["q"], p, case), out[0], out[2], out[1], out[3]
        o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full((H, o.shape[0]), -math.inf, dtype=torch.float64, device="cuda")
        for b, L in enumerate(st["lens"].tolist()):
            a, e = cu[b], cu[b + 1]
            ids = torch.tensor(table[b][:-(-L // block)], device="cuda")
            hidden = torch.arange(L, device="cuda")[None] > L - (e - a) + torch.arange(e - a, device="cuda")[:, None]
            for hk in range(Hk):
                k, v = ((c[ids, hk].double() * s[ids, hk].double()[:, None, None]).reshape(-1, d)[:L]
                        for c, s in ((st["ck"], st["sk"]), (st["cv"], st["sv"])))
                for h in range(hk * (H // Hk), (hk + 1) * (H // Hk)):
                    s = (st["q"][a:e, h].double() @ k.T) / math.sqrt(d)
                    if case["causal"]:
                        s[hidden] = -math.inf
                    lse[h, a:e] = torch.logsumexp(s, 1)
                    o[a:e, h] = torch.exp(s - lse[h, a:e, None]) @ v
        return o, lse
