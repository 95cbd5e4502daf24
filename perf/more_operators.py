"""The operators of the FP8 paged KV cache with a scale for each block and head, and rotary
positions, as cases that can be timed.

``run`` computes them in plain torch (``own`` false) or through the package's public calls
(``own`` true) on the same state:

  write   rows quantized into the cache by slot (block scales made as they are written), then
          read back by the same slots
  decode  one query per sequence over that cache
  multi   several query tokens per sequence over it: causal (the sequence's own last tokens) or
          not (cross attention: every query sees every cached token)
  rotary  query and key heads rotated by their positions

Block-scaled format: E4M3 codes uint8 [blocks][block_size][n_kv][head_dim], and a float32 scale
per block and kv head; an element is code * scale.  A write that holds a block's first token
starts the block anew; any other write keeps its scale or raises it, and the block's older codes
are then rounded to the new one.  A scale that a write makes is the smallest power of two (2^-60
at least) that takes the largest finite element to 448 or less.
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------- cases

def listed():
    attn = dict(op="decode", n_q=32, n_kv=8, hd=128, bs=16, spread=0.0)
    rot = dict(op="rotary", n_q=32, n_kv=8, hd=128, rot=128, layout="half", src="bf16", scaling="none",
               factor=1.0, longest=4096)
    return [
        # a serving step: one new token for each of 256 sequences, somewhere in its last block
        dict(name="write_step", op="write", seqs=256, run=1, append=True, n_kv=8, hd=128, bs=32, src="bf16", pad=0.0),
        # prompts of 16 sequences written at once, the last rows of each call padding
        dict(name="write_prompts", op="write", seqs=16, run=2048, append=False, n_kv=8, hd=128, bs=16, src="bf16",
             pad=0.03),
        # float32 rows of a small model: chunks that go on inside a block, an odd count of rows and of heads
        dict(name="write_f32_odd", op="write", seqs=7, run=585, append=True, n_kv=5, hd=64, bs=64, src="f32", pad=0.1),
        # the smallest serving step: four short sequences, latency only
        dict(attn, name="decode_tiny", seqs=4, n_q=4, n_kv=2, hd=64, longest=100, spread=0.8),
        # a full serving batch at equal lengths
        dict(attn, name="decode_batch", seqs=64, longest=4096),
        # few long ragged contexts
        dict(attn, name="decode_long", seqs=8, n_q=64, longest=131072, spread=0.75),
        # drafted tokens verified: four new tokens per sequence
        dict(attn, name="multi_verify", op="multi", seqs=32, longest=4099, spread=0.5, qlen=4, causal=True),
        # prompt chunks of 512 tokens
        dict(attn, name="multi_chunk", op="multi", seqs=16, longest=4096, spread=0.5, qlen=512, causal=True),
        # cross attention of decoder prompts to encoder states of another length
        dict(attn, name="multi_cross", op="multi", seqs=24, n_q=16, n_kv=16, hd=64, longest=1500, spread=0.3, qlen=225,
             causal=False),
        # a serving step's queries and keys at far positions, frequencies scaled by parts
        dict(rot, name="rotary_step", tokens=256, scaling="parts", factor=4.0, longest=131072),
        # prompts, pairs side by side in the first half of each head
        dict(rot, name="rotary_prompts", tokens=32768, rot=64, layout="interleaved"),
        # float32 heads of a small model, an odd count of tokens
        dict(rot, name="rotary_f32_odd", tokens=4099, n_q=14, n_kv=2, hd=64, rot=32, src="f32", scaling="linear",
             factor=2.0, longest=16384),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["write", "decode", "multi", "multi", "rotary", "decode", "write"])
    if op == "write":
        n_kv, hd = rng.choice([(2, 64), (8, 128), (4, 256), (1, 128), (5, 64), (16, 128)])
        tokens = _log(rng, 1, 32768 if n_kv * hd <= 1024 else 16384)
        seqs = max(1, min(256, _log(rng, 1, tokens)))
        return dict(op=op, seqs=seqs, run=max(1, tokens // seqs), append=rng.random() < 0.6, n_kv=n_kv, hd=hd,
                    bs=rng.choice([16, 32, 64, 128, 256]), src=rng.choice(["bf16", "f32"]), pad=rng.choice([0.0, 0.05]))
    if op in ("decode", "multi"):
        n_q, n_kv, hd = rng.choice([(32, 8, 128), (4, 2, 64), (64, 8, 128), (16, 16, 128), (16, 4, 256),
                                    (24, 8, 64), (14, 2, 64), (40, 8, 128), (16, 16, 64)])
        seqs = _log(rng, 1, 64)
        longest = _log(rng, 1, max(2, min(131072, 262144 // seqs)))
        c = dict(op=op, seqs=seqs, n_q=n_q, n_kv=n_kv, hd=hd, bs=rng.choice([16, 32, 64, 128]),
                 longest=longest, spread=rng.choice([0.0, 0.5, 0.9]))
        if op == "multi":
            c["causal"] = rng.random() < 0.6
            most = min(longest if c["causal"] else 512, 512, max(1, (1 << 27) // (seqs * longest * n_q // 8 + 1)))
            c["qlen"] = _log(rng, 1, most)
        return c
    n_q, n_kv, hd, rot = rng.choice([(32, 8, 128, 128), (4, 2, 64, 64), (64, 8, 128, 32), (16, 4, 256, 64),
                                     (14, 2, 64, 32), (40, 8, 128, 96), (5, 1, 80, 80), (16, 16, 64, 16)])
    return dict(op=op, tokens=_log(rng, 1, 32768 if (n_q + n_kv) * hd <= 5120 else 16384), n_q=n_q, n_kv=n_kv, hd=hd,
                rot=rot, layout=rng.choice(["half", "interleaved"]), src=rng.choice(["bf16", "f32"]),
                scaling=rng.choice(["none", "linear", "base", "parts"]), factor=rng.choice([2.0, 8.0]),
                longest=_log(rng, 64, 1 << 20))


# ---------------------------------------------------------------- what follows from a case alone

def _of(case):
    """A generator that goes by the case's sizes, not by the seed: lengths and which offsets are written."""
    return np.random.default_rng([ord(ch) for ch in "".join("%s=%s;" % (k, case[k]) for k in sorted(case) if k != "name")])


def _lens(case):
    r = _of(case)
    n, hi = case["seqs"], case["longest"]
    lens = np.maximum(1, np.round(hi * (1 - case["spread"] * r.random(n)))).astype(np.int64)
    lens[int(r.integers(n))] = hi
    return lens


def _qlens(case):
    """Query tokens per sequence: `qlen`, every third sequence fewer; causal ones are among what it holds."""
    if case["op"] == "decode":
        return np.ones(case["seqs"], np.int64)
    q = np.full(case["seqs"], case["qlen"], np.int64)
    q[2::3] = max(1, (2 * case["qlen"]) // 3)
    return np.minimum(q, _lens(case)) if case["causal"] else q


def _starts(case):
    """The offset of each sequence's first written token in its first block."""
    return _of(case).integers(0, case["bs"], case["seqs"]) if case["append"] else np.zeros(case["seqs"], np.int64)


def work(case):
    op, hd = case["op"], case["hd"]
    if op == "write":
        n, bs, row = case["seqs"] * case["run"], case["bs"], case["n_kv"] * hd
        n -= int(case["pad"] * n)
        blocks = int(np.sum(-(-(_starts(case) + case["run"]) // bs)))
        src = 4 if case["src"] == "f32" else 2
        # rows in, codes out, block scales in and out; codes in, 16-bit rows out
        return {"bytes": 2 * n * row * (src + 1 + 1 + 2) + 2 * blocks * case["n_kv"] * 12 + 16 * n, "flops": 0}
    if op in ("decode", "multi"):
        lens, q = _lens(case), _qlens(case)
        seen = float(np.sum(q * lens - (q * (q - 1) // 2 if case.get("causal", True) else 0)))  # (query, key) pairs
        blocks = float(np.sum(-(-lens // case["bs"])))
        return {"bytes": float(lens.sum()) * case["n_kv"] * hd * 2 + float(q.sum()) * case["n_q"] * hd * 4
                + blocks * (4 + 8 * case["n_kv"]) + 8 * len(lens),
                "flops": 4 * seen * case["n_q"] * hd}
    elems = case["tokens"] * (case["n_q"] + case["n_kv"]) * hd
    return {"bytes": 2 * elems * (4 if case["src"] == "f32" else 2) + 8 * case["tokens"] + 4 * case["rot"],
            "flops": 3 * elems * case["rot"] / hd}


# ---------------------------------------------------------------- inputs

def _normal(shape, std, gen, dtype):
    """Normal values, heads of different spread, a few outliers."""
    x = torch.randn(shape, generator=gen, device="cuda") * std
    x *= torch.exp2(torch.arange(shape[-2], device="cuda") % 5 - 2.0)[:, None]
    return torch.where(torch.rand(shape, generator=gen, device="cuda") < 1e-3, x * 20, x).to(dtype)


def _cache(blocks, bs, n_kv, hd, gen):
    """One side of a cache whose blocks are full: codes and block scales."""
    x = _normal((blocks, bs, n_kv, hd), 1.5, gen, torch.bfloat16)
    x *= torch.exp2(torch.randint(-2, 3, (blocks, 1, n_kv, 1), generator=gen, device="cuda").float()).to(x.dtype)
    scales = torch.zeros(blocks, -(-n_kv // 4) * 4, device="cuda")
    scales[:, :n_kv] = _power(x.abs().amax((1, 3)).float())
    return _encode(x.float() / scales[:, None, :n_kv, None]), scales


def _tables(case, rng, blocks):
    """Block tables [seqs, most blocks] of the lengths, unused entries -1, physical order shuffled."""
    need = -(-_lens(case) // case["bs"])
    bt = np.full((len(need), int(need.max())), -1, np.int32)
    bt[np.arange(bt.shape[1])[None, :] < need[:, None]] = rng.permutation(blocks)[:int(need.sum())]
    return bt


def _frequencies(case):
    """Radians per position of the rot / 2 pairs, in 64 bits, and what the rotated values are multiplied by."""
    rot, factor, base = case["rot"], case["factor"], 10000.0
    if case["scaling"] == "base":  # a larger base, so that the slowest pair turns `factor` times slower
        base *= factor ** (rot / max(2, rot - 2))
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "parts":  # pairs of few turns in the first 8192 positions slowed down, fast ones kept
        turns = 8192 * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    op, n_kv, hd = case["op"], case["n_kv"], case["hd"]
    dtype = torch.float32 if case.get("src") == "f32" else torch.bfloat16
    st = dict(case=case)
    if op == "write":
        bs, run, starts = case["bs"], case["run"], _starts(case)
        need = -(-(starts + run) // bs)
        blocks = int(need.sum()) + 2
        ids, slots, used = rng.permutation(blocks), [], 0
        for at, m in zip(starts, need):
            pos = at + np.arange(run)
            slots.append(ids[used + pos // bs] * bs + pos % bs)
            used += int(m)
        slots = np.concatenate(slots).astype(np.int64)
        n = len(slots)
        slots[n - int(case["pad"] * n):] = -1
        for side in "kv":
            st[side] = _normal((n, n_kv, hd), 1.5, gen, dtype)
            st[side + "c"], st[side + "s"] = _cache(blocks, bs, n_kv, hd, gen)
        st["slots"] = dev(slots)
        return st
    if op in ("decode", "multi"):
        bs, lens, q = case["bs"], _lens(case), _qlens(case)
        blocks = int(np.sum(-(-lens // bs))) + 3
        for side in "kv":
            st[side + "c"], st[side + "s"] = _cache(blocks, bs, n_kv, hd, gen)
        st.update(bt=dev(_tables(case, rng, blocks)), lens=dev(lens.astype(np.int32)),
                  q=(torch.randn((int(q.sum()), case["n_q"], hd), generator=gen, device="cuda") / 4).to(torch.bfloat16),
                  qsl=dev(np.concatenate([[0], np.cumsum(q)]).astype(np.int32)), qmax=int(q.max()))
        return st
    f, magnitude = _frequencies(case)
    for name, heads in (("q", case["n_q"]), ("k", n_kv)):
        st[name] = torch.randn((case["tokens"], heads, hd), generator=gen, device="cuda").to(dtype)
    st.update(pos=dev(rng.integers(0, case["longest"], case["tokens"])), f=dev(f), magnitude=magnitude)
    return st


# ---------------------------------------------------------------- the plain forms

def _encode(y):
    """float32 -> E4M3 codes, to nearest even, saturating."""
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _power(a):
    """The smallest power of two, 2^-60 at least, with 448 times it not below a (float32)."""
    m, e = torch.frexp(a)
    k = (e - 9 + (m > 0.875).int()).clamp(min=-60)
    return ((torch.where(a > 0, k, -60) + 127) << 23).view(torch.float32)


def _values(codes, scales):
    """Codes [blocks, bs, n_kv, hd] and block scales -> float32 values."""
    return codes.view(torch.float8_e4m3fn).float() * scales[:, None, :codes.shape[2], None]


def _plain_write(st, x, codes, scales):
    blocks, bs, n_kv, _ = codes.shape
    ok = st["slots"] >= 0
    rows, slots = x[ok].float(), st["slots"][ok]
    blk, off = slots // bs, slots % bs
    top = torch.zeros(blocks, n_kv, device="cuda")
    top.scatter_reduce_(0, blk[:, None].expand(-1, n_kv), rows.abs().amax(-1), "amax")
    fresh = torch.zeros(blocks, dtype=torch.bool, device="cuda")
    fresh[blk[off == 0]] = True
    ids = torch.unique(blk)
    old = scales[ids, :n_kv]
    new = torch.where(fresh[ids][:, None], 0.0, old).maximum(_power(top[ids]))
    raised = (new > old) & ~fresh[ids][:, None]
    held = codes[ids].view(torch.float8_e4m3fn).float()
    held = _encode(held * torch.where(raised, old / new, 1.0)[:, None, :, None])
    codes[ids] = torch.where(raised[:, None, :, None], held, codes[ids])
    scales[ids, :n_kv] = new
    codes[blk, off] = _encode(rows / scales[blk, :n_kv, None])
    out = torch.zeros(x.shape, device="cuda")
    out[ok] = codes[blk, off].view(torch.float8_e4m3fn).float() * scales[blk, :n_kv, None]
    return out.to(torch.bfloat16)


def _plain_attention(st):
    case = st["case"]
    n_kv, hd, n_q = case["n_kv"], case["hd"], case["n_q"]
    bt, lens, qsl = st["bt"].long().clamp(min=0), st["lens"].long(), st["qsl"].long()

    def rows(side):  # [seqs, n_kv, tokens, hd]
        v = st[side + "c"][bt].view(torch.float8_e4m3fn).float() * st[side + "s"][bt][:, :, None, :n_kv, None]
        return v.permute(0, 3, 1, 2, 4).flatten(2, 3)

    at = qsl[:-1, None] + torch.arange(st["qmax"], device="cuda")
    there = at < qsl[1:, None]
    at = at.clamp(max=st["q"].shape[0] - 1)
    q = st["q"][at].float()
    b, m = q.shape[:2]
    q = q.view(b, m, n_kv, n_q // n_kv, hd).permute(0, 2, 1, 3, 4).reshape(b, n_kv, -1, hd)
    p = torch.matmul(q, rows("k").transpose(-1, -2)).mul_(hd ** -0.5)
    p = p.view(b, n_kv, m, n_q // n_kv, -1)
    last = (lens - 1)[:, None].expand(-1, m)  # the last token a row sees
    if case.get("causal", True):
        last = lens[:, None] - there.sum(1)[:, None] + torch.arange(m, device="cuda")
    seen = torch.arange(p.shape[-1], device="cuda") <= last[:, :, None]
    p.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True)).view(b, n_kv, m * (n_q // n_kv), -1)
    o = torch.matmul(p, rows("v")).view(b, n_kv, m, n_q // n_kv, hd).permute(0, 2, 1, 3, 4)
    out = torch.empty_like(st["q"])
    out[at[there]] = o.reshape(b, m, n_q, hd)[there].to(torch.bfloat16)
    return out


def _pairs(x, rot, layout):
    """The two members of each pair of the first rot dims."""
    return (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])


def _plain_rotary(st, x):
    case = st["case"]
    angle = st["pos"].double()[:, None] * st["f"]
    cos, sin = (torch.cos(angle) * st["magnitude"]).float()[:, None], (torch.sin(angle) * st["magnitude"]).float()[:, None]
    out = x.to(torch.float32, copy=True)
    a, b = _pairs(out, case["rot"], case["layout"])
    a2, b2 = a * cos - b * sin, a * sin + b * cos
    a.copy_(a2)
    b.copy_(b2)
    return out.to(x.dtype)


def _as_values(codes):
    return codes.view(torch.float8_e4m3fn)


def run(st):
    case = st["case"]
    op = case["op"]
    if own:
        import fp8_paged_kv_reshape_gb300 as kv
    if op == "write":
        if own:
            kv.reshape_and_cache_block_scaled(st["k"], st["v"], st["kc"], st["vc"], st["ks"], st["vs"], st["slots"])
            k = kv.dequant_block_scaled(st["kc"], st["ks"], st["slots"], torch.bfloat16)
            v = kv.dequant_block_scaled(st["vc"], st["vs"], st["slots"], torch.bfloat16)
        else:
            k = _plain_write(st, st["k"], st["kc"], st["ks"])
            v = _plain_write(st, st["v"], st["vc"], st["vs"])
        return {"k": k, "v": v, "kc": _as_values(st["kc"]), "vc": _as_values(st["vc"]), "ks": st["ks"], "vs": st["vs"]}
    if op == "decode":
        if own:
            return kv.paged_decode_attention_block_scaled(st["q"], st["kc"], st["vc"], st["ks"], st["vs"], st["bt"],
                                                          st["lens"])
        return _plain_attention(st)
    if op == "multi":
        if own:
            return kv.paged_attention_multi_block_scaled(st["q"], st["qsl"], st["qmax"], st["kc"], st["vc"], st["ks"],
                                                         st["vs"], st["bt"], st["lens"], causal=case["causal"])
        return _plain_attention(st)
    if own:
        return kv.rotary_embedding(st["q"], st["k"], st["pos"], st["f"], interleaved=case["layout"] == "interleaved",
                                   magnitude=st["magnitude"])
    return _plain_rotary(st, st["q"]), _plain_rotary(st, st["k"])


# ---------------------------------------------------------------- 64 bits, from the definition

def _e4m3(device="cuda"):
    """The 127 values of E4M3 that are not negative, ascending, float64."""
    return torch.tensor([m * 2.0 ** -9 if e == 0 else 2.0 ** (e - 7) * (1 + m / 8)
                         for e in range(16) for m in range(8)][:127], dtype=torch.float64, device=device)


def _decoded(codes):
    """Codes -> float64 code values, by table."""
    table = _e4m3()
    table = torch.cat([table, table.new_tensor([float("nan")])])
    return torch.cat([table, -table])[codes.int()]


def _rounded(y):
    """float64 -> the nearest E4M3 value (halfway to the even code), saturating."""
    levels = _e4m3()
    x = y.abs().contiguous()
    i = torch.searchsorted(levels, x, right=True).clamp(1, len(levels) - 1)
    lo, hi = levels[i - 1], levels[i]
    up = (x - lo > hi - x) | ((x - lo == hi - x) & (i % 2 == 0))
    return torch.where(up, hi, lo).copysign(y)


def _exact_written(x, slots, codes, scales):
    bs, n_kv = codes.shape[1], codes.shape[2]
    cache, scale = _decoded(codes), scales.double()
    rows = x.double()
    slots = slots.cpu().numpy()
    there = np.nonzero(slots >= 0)[0]
    order = there[np.argsort(slots[there], kind="stable")]  # by slot, so by block
    blk = slots[order] // bs
    first = np.nonzero(np.r_[True, blk[1:] != blk[:-1]])[0]
    group = torch.from_numpy(np.repeat(np.arange(len(first)), np.diff(np.r_[first, len(blk)]))).cuda()
    ids = torch.from_numpy(blk[first]).cuda()
    starts_anew = torch.from_numpy(slots[order][first] % bs == 0).cuda()
    src, dst = torch.from_numpy(order).cuda(), torch.from_numpy(slots[order]).cuda()
    top = rows[src].abs().amax(-1)
    top = torch.zeros(len(first), n_kv, dtype=torch.float64, device="cuda").index_reduce_(0, group, top, "amax")
    k = torch.full_like(top, -60.0)
    for e in range(-60, 121):  # the smallest exponent that holds the largest element
        k = torch.where(top > 448.0 * 2.0 ** (e - 1), max(e, -60), k)
    old = torch.where(starts_anew[:, None], 0.0, scale[ids, :n_kv])
    new = torch.maximum(old, torch.exp2(k))
    grown = (new > old) & (old > 0)
    held = cache[ids] * torch.where(grown, old / new, torch.ones_like(new))[:, None, :, None]
    cache[ids] = torch.where(grown[:, None, :, None], _rounded(held), held)
    scale[ids, :n_kv] = new
    s = new[group][:, :, None]
    flat = cache.view(-1, n_kv, cache.shape[3])
    flat[dst] = _rounded((rows[src] / s).float().double())  # quotients are float quotients
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    out[src] = flat[dst] * s
    return out, cache, scale


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "write":
        got = {}
        for side in "kv":
            got[side], got[side + "c"], got[side + "s"] = _exact_written(st[side], st["slots"], st[side + "c"],
                                                                         st[side + "s"])
        return {name: got[name] for name in ("k", "v", "kc", "vc", "ks", "vs")}
    if op in ("decode", "multi"):
        bs, n_kv, hd, group = case["bs"], case["n_kv"], case["hd"], case["n_q"] // case["n_kv"]
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        qsl = st["qsl"].tolist()
        for i, length in enumerate(st["lens"].tolist()):
            t = torch.arange(length, device="cuda")
            b, o = st["bt"][i].long()[t // bs], t % bs
            q = st["q"][qsl[i]:qsl[i + 1]].double()
            for h in range(n_kv):
                kh = _decoded(st["kc"][b, o, h]) * st["ks"][b, h].double()[:, None]
                vh = _decoded(st["vc"][b, o, h]) * st["vs"][b, h].double()[:, None]
                x = (q[:, h * group:(h + 1) * group].reshape(-1, hd) @ kh.t()) / math.sqrt(hd)
                x = x.view(len(q), group, length)
                if case.get("causal", True):
                    at = torch.arange(length - len(q), length, device="cuda")
                    x = x.masked_fill(t > at[:, None, None], float("-inf"))
                out[qsl[i]:qsl[i + 1], h * group:(h + 1) * group] = torch.softmax(x, -1) @ vh
        return out
    # the complex number of each pair, turned
    f, magnitude = _frequencies(case)
    turn = torch.polar(torch.full((case["tokens"], case["rot"] // 2), magnitude, dtype=torch.float64, device="cuda"),
                       torch.remainder(st["pos"].double()[:, None] * torch.from_numpy(f).cuda(), 2 * math.pi))

    def turned(x):
        x = x.double()
        a, b = _pairs(x, case["rot"], case["layout"])
        z = torch.complex(a.contiguous(), b.contiguous()) * turn[:, None]
        if case["layout"] == "half":
            return torch.cat([z.real, z.imag, x[..., case["rot"]:]], -1)
        return torch.cat([torch.view_as_real(z).flatten(-2), x[..., case["rot"]:]], -1)

    return turned(st["q"]), turned(st["k"])
