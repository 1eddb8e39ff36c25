"""Cases and plain forms of the operators that extend a cached prompt.

Three operators of the paged quantised KV cache, as a server calls them when a
prompt grows a cached prefix:

  append   rotate the chunk's queries and keys by their positions (one or more
           axes), quantise keys and values into the paged cache as they are
           written, and read the written rows back as the values they stand for
  gather   read ranges of cached tokens back through the block tables
  attend   attention of a chunk of new tokens over the paged cache: causal among
           the new tokens, remapped slots with logit -1e4 and value 0

`run` computes them in plain torch where `own` is false and calls the package
where it is true.  Shapes follow the cache's own workloads (Gemma 3 12B: 16/8
heads of 256, bf16; Llama 3.1 8B: 32/8 of 128, fp16; Qwen2.5-14B: 40/8 of 128,
fp16, 60 % of the slots remapped).
"""
import math
import random

import torch

own = False

BLOCK, GROUP = 256, 64
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# -- cases -------------------------------------------------------------------

def _attend(name, B, T, ctx, hq, hkv, d, dtype, n8=0.0, n2=0.0, fp8=False, rotated=True, evict=0.0, window=0, ragged=0):
    return dict(name=name, op="attend", B=B, T=T, ctx=ctx, hq=hq, hkv=hkv, d=d, dtype=dtype, n8=n8, n2=n2, fp8=fp8,
                rotated=rotated, evict=evict, window=window, ragged=ragged)


def _append(name, B, T, ctx, hq, hkv, d, dtype, bits=4, rotated=True, rot=128, axes=1, interleaved=False, given=False,
            unrotate=False, ragged=0):
    return dict(name=name, op="append", B=B, T=T, ctx=ctx, hq=hq, hkv=hkv, d=d, dtype=dtype, bits=bits, rotated=rotated,
                rot=rot, axes=axes, interleaved=interleaved, given=given, unrotate=unrotate, ragged=ragged)


def _gather(name, B, ctx, hkv, d, dtype, n8=0.0, n2=0.0, fp8=False, rotated=True, evict=0.0, unrotate=False, ragged=0):
    return dict(name=name, op="gather", B=B, ctx=ctx, hkv=hkv, d=d, dtype=dtype, n8=n8, n2=n2, fp8=fp8, rotated=rotated,
                evict=evict, unrotate=unrotate, ragged=ragged)


def listed():
    return [
        # a drafted run of four tokens checked against one short session
        _attend("attend_verify_1x4_1k", 1, 4, 1020, 32, 8, 128, "fp16"),
        # drafted runs of five tokens of sixteen long sessions, ragged
        _attend("attend_verify_16x5_32k", 16, 5, 32768, 32, 8, 128, "fp16", ragged=1),
        # turns of up to 509 tokens on four evicted sessions
        _attend("attend_turn_4x509_evict", 4, 509, 16384, 40, 8, 128, "fp16", evict=0.6, ragged=2),
        # turns on five sessions of heads of 256
        _attend("attend_turn_5x256_d256", 5, 256, 8192, 16, 8, 256, "bf16", ragged=3),
        # a long document chunk on a long mixed 4/8-bit prefix
        _attend("attend_chunk_1x2048_32k", 1, 2048, 32768, 32, 8, 128, "bf16", n8=0.25),
        # fresh prompts, windowed layer of the FP8 comparison cache
        _attend("attend_prompt_3x1500_win", 3, 1500, 0, 16, 8, 256, "bf16", fp8=True, rotated=False, window=1024, ragged=4),
        # the step of one new token for thirty-two sessions
        _append("append_step_32x1", 32, 1, 16384, 40, 8, 128, "fp16"),
        # a prompt chunk with heads of 256, half of each rotated
        _append("append_chunk_1x8191_d256", 1, 8191, 1000, 16, 8, 256, "bf16", rot=128),
        # images: three position axes, adjacent pairs, ragged prompts
        _append("append_image_4x2048_axes3", 4, 2048, 333, 32, 8, 128, "fp16", rot=128, axes=3, interleaved=True, given=True,
                unrotate=True, ragged=5),
        # one short session read back
        _gather("gather_1x1000", 1, 1000, 8, 128, "fp16"),
        # ten mixed 4/8-bit sessions handed off, keys un-rotated
        _gather("gather_10x32768_mixed", 10, 32768, 8, 128, "fp16", n8=0.25, unrotate=True),
        # five ragged sessions with heads of 256, some slots remapped
        _gather("gather_5x8192_d256", 5, 8192, 8, 256, "bf16", evict=0.3, unrotate=True, ragged=6),
    ]


HEADS = ((32, 8, 128), (40, 8, 128), (16, 8, 256), (8, 8, 128), (12, 3, 128), (16, 2, 256))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attend", "attend", "append", "gather"))
    hq, hkv, d = rng.choice(HEADS)
    dtype = rng.choice(("fp16", "bf16"))
    ragged = rng.randrange(1, 1000)
    if op == "attend":
        ctx, B = _log(rng, 1, 32768) - 1, _log(rng, 1, 16)
        most = min(2048, max(1, 2048 * 32 * 34816 // (B * hq * (ctx + 2048))))
        T = _log(rng, 1, most)
        kind = rng.choice(("4", "4", "48", "482", "fp8"))
        return _pure(_attend("", B, T, ctx, hq, hkv, d, dtype, n8=0.25 if "8" in kind else 0.0, n2=0.25 if "2" in kind else 0.0,
                             fp8=kind == "fp8", rotated=kind != "fp8" and rng.random() < 0.8, evict=rng.choice((0.0, 0.0, 0.6)),
                             window=rng.choice((0, 0, 0, _log(rng, 16, 4096))), ragged=ragged))
    if op == "append":
        B = _log(rng, 1, 32)
        rot = rng.choice((d, d, d // 2, 64))
        axes = rng.choice((1, 1, 2, 3))
        return _pure(_append("", B, _log(rng, 1, max(1, 8192 // B)), _log(rng, 1, 16384) - 1, hq, hkv, d, dtype,
                             bits=rng.choice((4, 4, 8, 2)), rotated=rng.random() < 0.8, rot=rot, axes=axes,
                             interleaved=rng.random() < 0.5, given=axes > 1 or rng.random() < 0.3, unrotate=rng.random() < 0.5,
                             ragged=ragged))
    B = _log(rng, 1, 16)
    kind = rng.choice(("4", "48", "482", "fp8"))
    return _pure(_gather("", B, _log(rng, 1, min(32768, 10 * 32768 // B)), hkv, d, dtype, n8=0.25 if "8" in kind else 0.0,
                         n2=0.25 if "2" in kind else 0.0, fp8=kind == "fp8", rotated=kind != "fp8" and rng.random() < 0.8,
                         evict=rng.choice((0.0, 0.3)), unrotate=rng.random() < 0.5, ragged=ragged))


def _pure(case):
    return {k: v for k, v in case.items() if k != "name"}


def _lengths(c):
    """Per sequence: cached tokens before the call, new (or read) tokens, first token read."""
    r, B = random.Random(c["ragged"]), c["B"]
    if c["op"] == "gather":
        start = [r.randrange(0, c["ctx"] // 2 + 1) if c["ragged"] else 0 for _ in range(B)]
        return [0] * B, [c["ctx"] - s for s in start], start
    lens = [r.randrange(c["ctx"] // 2, c["ctx"] + 1) if c["ragged"] and b else c["ctx"] for b in range(B)]
    new = [r.randrange((c["T"] + 1) // 2, c["T"] + 1) if c["ragged"] and b else c["T"] for b in range(B)]
    return lens, new, lens


def work(c):
    lens, new, _ = _lengths(c)
    hkv, d, n = c["hkv"], c["d"], sum(new)
    if c["op"] == "append":
        bits, e = c["bits"], hkv * d * 2 * 2
        row = hkv * 2 * (d * bits / 8 + d // GROUP * 4)
        # q, k and v read, q written, the cache written and read back, the values written
        return {"bytes": n * (2 * c["hq"] * d * 2 + e + 2 * row + e + 4 * c["rot"]), "flops": n * (c["hq"] + hkv) * c["rot"] * 3}
    n8, n2 = (1.0, 0.0) if c["fp8"] else (c["n8"], c["n2"])
    bits = 8 * n8 + 2 * n2 + 4 * (1 - n8 - n2)
    row = hkv * 2 * (d * bits / 8 + (0 if c["fp8"] else d // GROUP * 4))
    live = 1 - c["evict"]
    if c["op"] == "gather":
        return {"bytes": n * (row * live + hkv * d * 4), "flops": n * hkv * d * 4}
    seen, read = 0, 0
    for a, t in zip(lens, new):
        w = c["window"] or a + t
        seen += sum(min(a + i + 1, w) for i in range(t))
        read += min(a + t, w + t - 1) if t else 0
    return {"bytes": read * row * live + 2 * n * c["hq"] * d * 2, "flops": 4 * d * c["hq"] * seen * live}


# -- inputs ------------------------------------------------------------------

def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 1000003 + 17)
    lens, new, start = _lengths(c)
    B, hkv, d = c["B"], c["hkv"], c["d"]
    dt = DTYPES[c["dtype"]]
    nb = max(1, -(-max(a + t for a, t in zip(start, new)) // BLOCK))
    n = B * nb
    s = {"case": c, "n_tokens": sum(new)}

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    fp8 = c.get("fp8", False)
    if c["op"] == "append":
        n8, n2 = (n if c["bits"] == 8 else 0), (n if c["bits"] == 2 else 0)
    else:
        n8, n2 = (n if fp8 else int(n * c["n8"])), int(n * c["n2"])
    n4 = n - n8 - n2
    pool = {"k_rotated": c["rotated"], "fp8": fp8, "n": (n4, n8, n2)}
    for bits, m in ((4, n4), (8, n8), (2, n2)):
        if not m:
            continue
        for name in "kv":
            x = normal(m, hkv, BLOCK, d)
            x[..., 5::41] *= 8.0 if name == "k" and not c["rotated"] else 1.0   # outlier channels of raw keys
            if fp8:
                pool[name + "_codes8"] = x.to(torch.float8_e4m3fn).view(torch.uint8)
            else:
                codes, params = encode(x, bits)
                pool["%s_codes%d" % (name, bits)], pool["%s_params%d" % (name, bits)] = codes, params
    gone = torch.rand((n, 8, 32), generator=g, device=dev) < c.get("evict", 0.0)
    words = (gone.to(torch.int64) << torch.arange(32, device=dev)).sum(-1)
    pool["mask"] = (words - (words >> 31 << 32)).to(torch.int32)
    s["pool"] = pool
    s["tables"] = torch.randperm(n, generator=g, device=dev).view(B, nb).to(torch.int32)
    offsets = [sum(new[:b]) for b in range(B + 1)]
    s["offsets"], s["starts"] = ints(offsets), ints(start)
    s["rows"] = torch.cat([torch.arange(t, device=dev) + b * c.get("T", 0) for b, t in enumerate(new)])
    s["where"] = torch.cat([torch.arange(a, a + t, device=dev) + b * nb * BLOCK for b, (a, t) in enumerate(zip(start, new))])
    if c["op"] == "gather":
        return s
    T, hq = c["T"], c["hq"]
    s["seq_lens"] = ints(lens)
    s["n_new"] = ints(new) if c["ragged"] else None
    # q, k and v as the projection leaves them: slices of one row per token
    qkv = normal(B, T, hq + 2 * hkv, d).to(dt)
    s["q"], s["k"], s["v"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
    if c["op"] == "attend":
        s["q"] = s["q"].contiguous()
        # the session whose every slot is remapped answers zeros
        if c["evict"] and B > 2:
            pool["mask"][s["tables"][B - 1].long()] = -1
        return s
    half, axes = c["rot"] // 2, c["axes"]
    top = max(a + t for a, t in zip(lens, new))
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
    angle = torch.arange(top, dtype=torch.float64, device=dev)[:, None] * inv
    s["table"] = torch.stack((angle.cos(), angle.sin()), -1).float()
    s["axis"] = [f * axes // half for f in range(half)]
    s["axis_t"] = torch.tensor(s["axis"], device=dev)
    s["positions"] = torch.randint(0, top, (axes, B, T), generator=g, device=dev, dtype=torch.int32) if c["given"] else None
    return s


# -- plain forms -------------------------------------------------------------

def hadamard(x):
    """c H x along the last axis: butterflies of strides 1, 2, ..., D/2, one rounding each, then times c."""
    shape, d = x.shape, x.shape[-1]
    for e in range(d.bit_length() - 1):
        y = x.reshape(*shape[:-1], d >> (e + 1), 2, 1 << e)
        a, b = y[..., 0, :], y[..., 1, :]
        x = torch.stack((a + b, a - b), -2).reshape(shape)
    return x * torch.tensor(1.0 / math.sqrt(d), dtype=torch.float32).item()


def encode(x, bits):
    """Packed codes and (scale, zero) of groups of 64."""
    top = float(2 ** bits - 1)
    y = x.reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = y.amin(-1, keepdim=True) + 0.0, y.amax(-1, keepdim=True) + 0.0
    # by a tensor: torch divides by a number as a product with its reciprocal, which rounds otherwise
    s16, z16 = ((hi - lo) / torch.full_like(hi, top)).half(), lo.half()
    s, z = s16.float(), z16.float()
    codes = torch.where(s == 0, 0.0, ((y - z) / torch.where(s == 0, 1.0, s)).round().clamp(0, top)).to(torch.uint8)
    per = 8 // bits
    codes = codes.reshape(*x.shape[:-1], -1, per) << torch.arange(0, 8, bits, device=x.device, dtype=torch.uint8)
    return codes.sum(-1, dtype=torch.uint8), torch.cat((s16, z16), -1)


def decode(codes, params, bits):
    shift = torch.arange(0, 8, bits, device=codes.device, dtype=torch.uint8)
    x = ((codes[..., None] >> shift) & (2 ** bits - 1)).reshape(*params.shape[:-1], GROUP).float()
    return (x * params[..., :1].float() + params[..., 1:].float()).flatten(-2)


def rows_of(pool, name, blk, slot):
    """Values [n][Hkv][D] in 32 bits of slots `slot` of blocks `blk`."""
    n4, n8, n2 = pool["n"]
    if pool["fp8"]:
        return pool[name + "_codes8"][blk, :, slot].view(torch.float8_e4m3fn).float()
    x = None
    for n, first, bits in ((n4, 0, 4), (n8, n4, 8), (n2, n4 + n8, 2)):
        if n:
            at = (blk - first).clamp(0, n - 1)
            y = decode(pool["%s_codes%d" % (name, bits)][at, :, slot], pool["%s_params%d" % (name, bits)][at, :, slot], bits)
            x = y if x is None else torch.where((blk >= first)[:, None, None], y, x)
    return x


def gone_of(pool, blk, slot):
    """Which of the slots are remapped."""
    return ((pool["mask"][blk, slot // 32] >> (slot % 32).int()) & 1) == 1


def read_back(s, unrotate, dtype):
    """Keys and values of the case's tokens, packed [n][Hkv][D]."""
    pool, at = s["pool"], s["where"]
    blk, slot = s["tables"].flatten()[at // BLOCK].long(), at % BLOCK
    k, v = rows_of(pool, "k", blk, slot), rows_of(pool, "v", blk, slot)
    if unrotate and pool["k_rotated"]:
        k = hadamard(k)
    gone = gone_of(pool, blk, slot)[:, None, None]
    return [torch.where(gone, -1.0e4, k).to(dtype), torch.where(gone, 0.0, v).to(dtype)]


def rotate(s, x):
    """Rotary positions of rows [B][T][H][D], rounded once to their type."""
    c, r = s["case"], s["case"]["rot"]
    B, T = x.shape[:2]
    if s["positions"] is None:
        p = (s["seq_lens"][:, None].long() + torch.arange(T, device=x.device))[None].expand(c["axes"], B, T)
    else:
        p = s["positions"].long()
    p = p.clamp(max=s["table"].shape[0] - 1)[s["axis_t"]]                       # [pairs][B][T]
    cs = s["table"][p, torch.arange(r // 2, device=x.device)[:, None, None]].permute(1, 2, 0, 3)[:, :, None]
    cos, sin = cs[..., 0], cs[..., 1]
    y = x.float()
    at = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
    a, b = y[..., at[0]], y[..., at[1]]
    out = y.clone()
    out[..., at[0]], out[..., at[1]] = a * cos - b * sin, b * cos + a * sin
    return out.to(x.dtype)


def plain_append(s):
    c, pool = s["case"], s["pool"]
    dt, bits = DTYPES[c["dtype"]], c["bits"]
    k, v = rotate(s, s["k"]).float(), s["v"].float()
    if pool["k_rotated"]:
        k = hadamard(k)
    at = s["where"]
    blk = s["tables"].flatten().long()[at // BLOCK]
    slot = at % BLOCK
    for name, x in (("k", k), ("v", v)):
        codes, params = encode(x.flatten(0, 1)[s["rows"]], bits)
        pool["%s_codes%d" % (name, bits)][blk, :, slot] = codes
        pool["%s_params%d" % (name, bits)][blk, :, slot] = params
    q = rotate(s, s["q"])
    keep = torch.zeros(q.shape[0] * q.shape[1], dtype=torch.bool, device=q.device).index_fill(0, s["rows"], True)
    q = torch.where(keep.view(*q.shape[:2], 1, 1), q, 0.0).to(dt)
    return [q] + read_back(s, c["unrotate"], dt)


def plain_attend(s):
    c, pool = s["case"], s["pool"]
    B, T, hq, hkv, d = c["B"], c["T"], c["hq"], c["hkv"], c["d"]
    C = s["tables"].shape[1] * BLOCK
    at = torch.arange(C, device=s["q"].device)
    blk, slot = s["tables"].long().repeat_interleave(BLOCK, 1).flatten(), (at % BLOCK).repeat(B)
    gone = gone_of(pool, blk, slot)
    k = rows_of(pool, "k", blk, slot)
    v = torch.where(gone[:, None, None], 0.0, rows_of(pool, "v", blk, slot))
    k, v = (x.view(B, C, hkv, d).transpose(1, 2) for x in (k, v))
    q = s["q"].float()
    if pool["k_rotated"]:
        q = hadamard(q)
    q = q.view(B, T, hkv, -1, d).transpose(1, 2).reshape(B, hkv, -1, d)         # rows (token, head of the group)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(d ** -0.5)
    x.masked_fill_(gone.view(B, 1, 1, C), -1.0e4)
    i = torch.arange(T, device=x.device).repeat_interleave(hq // hkv)
    p = s["seq_lens"][:, None].long() + i                                       # [B][rows]
    hidden = at > p[..., None]
    if c["window"]:
        hidden |= at <= p[..., None] - c["window"]
    x.masked_fill_(hidden[:, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(x, v) / x.sum(-1, keepdim=True)
    if s["n_new"] is not None:
        o = torch.where((i < s["n_new"][:, None])[:, None, :, None], o, 0.0)
    return o.view(B, hkv, T, -1, d).transpose(1, 2).reshape(B, T, hq, d).to(DTYPES[c["dtype"]])


# -- one pass ----------------------------------------------------------------

def _handles(s):
    """What a program keeps beside its tensors: the pool, the rotary description, the plan and its scratch."""
    import decode_attention_q4kv_b200 as q4

    if "handles" not in s:
        c, p = s["case"], s["pool"]
        pool = q4.Q4KVPool.from_tensors(c["hkv"], c["d"], k_rotated=p["k_rotated"], fp8=p["fp8"],
                                        **{k: v for k, v in p.items() if isinstance(v, torch.Tensor)})
        h = {"q4": q4, "pool": pool}
        if c["op"] == "append":
            h["rotary"] = q4.Rotary(s["table"], axis_of_pair=s["axis"], interleaved=c["interleaved"])
        if c["op"] == "attend":
            h["plan"] = q4.ExtendPlan(c["B"], c["T"], c["hq"], c["hkv"], c["d"], s["tables"].shape[1], window=c["window"])
            h["workspace"] = h["plan"].workspace(s["q"].device)
        s["handles"] = h
    return s["handles"]


def run(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if own:
        h = _handles(s)
        pool = h["pool"]
        if c["op"] == "attend":
            return h["q4"].extend_attention(pool, s["q"], s["tables"], s["seq_lens"], s["n_new"], window=c["window"], out_dtype=dt,
                                            plan=h["plan"], workspace=h["workspace"])
        if c["op"] == "append":
            q = pool.append_rotary(s["k"], s["v"], h["rotary"], s["tables"], s["seq_lens"], n_new=s["n_new"],
                                   positions=s["positions"], q=s["q"])
            return [q, *pool.gather(s["tables"], s["starts"], s["offsets"], s["n_tokens"], out_dtype=dt, unrotate_k=c["unrotate"])]
        return list(pool.gather(s["tables"], s["starts"], s["offsets"], s["n_tokens"], out_dtype=dt, unrotate_k=c["unrotate"]))
    if c["op"] == "attend":
        return plain_attend(s)
    return plain_append(s) if c["op"] == "append" else read_back(s, c["unrotate"], dt)


# -- the definition in 64 bits -----------------------------------------------

def _unit(d, dev):
    """H / sqrt(D) by the parity of the bits that row and column number share."""
    i = torch.arange(d, device=dev)
    both, parity = i[:, None] & i, torch.zeros(d, d, dtype=torch.int64, device=dev)
    for e in range(8):
        parity = parity ^ ((both >> e) & 1)
    return (1.0 - 2.0 * parity.double()) / math.sqrt(d)


def _block64(pool, blk, name):
    """Values of one block [Hkv][256][D] in 64 bits."""
    n4, n8, _ = pool["n"]
    bits, at = (4, blk) if blk < n4 else (8, blk - n4) if blk < n4 + n8 else (2, blk - n4 - n8)
    codes = pool["%s_codes%d" % (name, bits)][at].long()
    if pool["fp8"]:
        e, m = ((codes >> 3) & 15).double(), (codes & 7).double()
        mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2(e - 7))
        return torch.where(codes >= 128, -mag, mag)
    code = torch.stack([(codes // 2 ** (bits * j)) % 2 ** bits for j in range(8 // bits)], -1).flatten(-2).double()
    par = pool["%s_params%d" % (name, bits)][at].double().repeat_interleave(GROUP, -2)
    return code * par[..., 0] + par[..., 1]


def _tokens64(s, b, name):
    """Sequence b's cached rows [tokens][Hkv][D], and which are remapped."""
    ids = s["tables"][b].tolist()
    rows = torch.cat([_block64(s["pool"], i, name).transpose(0, 1) for i in ids])
    m = s["pool"]["mask"][ids].to(torch.int64)
    gone = torch.stack([(m >> j) & 1 for j in range(32)], -1).flatten() == 1
    return rows, gone


def _quantised64(x, bits):
    """What groups of 64 stand for once coded, from values in 64 bits."""
    y = x.unflatten(-1, (-1, GROUP))
    lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
    s, z = ((hi - lo) / (2 ** bits - 1)).half().double(), lo.half().double()
    code = torch.where(s > 0, torch.clamp(torch.round((y - z) / s.clamp(min=1e-300)), 0, 2 ** bits - 1), 0.0)
    return (code * s + z).flatten(-2)


def _rotated64(s, x, b, t):
    c, half = s["case"], s["case"]["rot"] // 2
    if s["positions"] is None:
        p = torch.arange(t, device=x.device) + int(s["seq_lens"][b])
        p = p[:, None].expand(t, half)
    else:
        p = torch.stack([s["positions"][a, b, :t].long() for a in s["axis"]], -1)
    cs = s["table"].double()[p, torch.arange(half, device=x.device)]
    z = torch.complex(cs[..., 0], cs[..., 1])[:, None]
    y = x[b, :t].double()
    r = y[..., :2 * half]
    pair = r.unflatten(-1, (half, 2)) if c["interleaved"] else r.unflatten(-1, (2, half)).transpose(-1, -2)
    w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
    w = w.flatten(-2) if c["interleaved"] else w.transpose(-1, -2).flatten(-2)
    return torch.cat((w, y[..., 2 * half:]), -1)


def exact(c, seed):
    s = prepare(c, seed)
    lens, new, start = _lengths(c)
    dev = s["tables"].device
    H = _unit(c["d"], dev)
    turn = c.get("unrotate", False) and c["rotated"]
    if c["op"] == "gather":
        out = ([], [])
        for b, (a, t) in enumerate(zip(start, new)):
            for which, name in enumerate("kv"):
                x, gone = _tokens64(s, b, name)
                x = x @ H if turn and name == "k" else x
                x[gone] = -1.0e4 if name == "k" else 0.0
                out[which].append(x[a:a + t])
        return [torch.cat(x) for x in out]
    if c["op"] == "append":
        q = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
        ks, vs = [], []
        for b, t in enumerate(new):
            q[b, :t] = _rotated64(s, s["q"], b, t)
            k = _rotated64(s, s["k"], b, t).to(s["k"].dtype).double()
            k = _quantised64(k @ H if c["rotated"] else k, c["bits"])
            ks.append(k @ H if turn else k)
            vs.append(_quantised64(s["v"][b, :t].double(), c["bits"]))
        return [q, torch.cat(ks), torch.cat(vs)]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    g = c["hq"] // c["hkv"]
    for b, (a, t) in enumerate(zip(lens, new)):
        (k, gone), (v, _) = _tokens64(s, b, "k"), _tokens64(s, b, "v")
        k, v, gone = k[:a + t], v[:a + t], gone[:a + t]
        v[gone] = 0.0
        at, p = torch.arange(a + t, device=dev), torch.arange(a, a + t, device=dev)[:, None]
        seen = (at <= p) & (at > p - (c["window"] or a + t + 1))
        for h in range(c["hq"]):
            q = s["q"][b, :t, h].double()
            x = (q @ H if c["rotated"] else q) @ k[:, h // g].T / math.sqrt(c["d"])
            x = x.masked_fill(gone, -1.0e4).masked_fill(~seen, -math.inf)
            out[b, :t, h] = torch.softmax(x, -1) @ v[:, h // g]
    return out
