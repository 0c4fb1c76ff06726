"""Cases for the operators around a prompt and an 8-bit latent cache.

Three operators are measured, each on seeded synthetic inputs:

  prefill   ``mlra_prefill``: causal attention of packed prompt tokens over
            the paged latent cache, every branch on its own
  decode8   ``mlra_decode_fp8``: one new token per sequence over a latent cache
            held as e4m3 values with one fp32 scale for each 16 tokens of a
            page and branch
  append8   ``mlra_append_fp8``: a run of new tokens per sequence written into
            that cache (scales found, values rounded, RoPE keys rotated)

``own`` False computes them with elementary torch operations, True calls the
library.  ``exact`` states each operator again in 64 bits.
"""
import math
import random

import torch

own = False

BLOCK = 16  # tokens that share one scale of the 8-bit cache, per branch
TOP = 448.0  # the largest e4m3 value


# ----------------------------------------------------------------- the cases
def listed():
    m29 = dict(heads=16, branches=4, d_c=128, d_r=64, page=64)   # the 2.9B-scale model shape
    tiny = dict(heads=8, branches=4, d_c=64, d_r=32, page=64)    # the tiny correctness shape
    mla = dict(heads=16, branches=1, d_c=512, d_r=64, page=64)   # one 512-wide branch (MLA)
    mla2 = dict(heads=16, branches=2, d_c=256, d_r=64, page=64)  # two 256-wide branches
    return [
        # a short question to a small model: the latency of one call
        dict(name="prompt_short", op="prefill", **tiny, n=1, new_lo=37, new_hi=37, past_lo=0, past_hi=0, mix=1),
        # a scheduler's batch of waiting prompts, from one token to a thousand, packed
        dict(name="prompt_packed", op="prefill", **m29, n=12, new_lo=1, new_hi=1024, past_lo=0, past_hi=0, mix=2),
        # one long prompt, the largest case
        dict(name="prompt_8k", op="prefill", **m29, n=1, new_lo=8192, new_hi=8192, past_lo=0, past_hi=0, mix=3),
        # chunked prefill: four prompts, each at its next 512 tokens
        dict(name="prompt_chunk", op="prefill", **m29, n=4, new_lo=512, new_hi=512, past_lo=7000, past_hi=7680, mix=4),
        # two odd-sized prompts of an MLA model
        dict(name="prompt_mla", op="prefill", **mla, n=2, new_lo=1900, new_hi=2001, past_lo=0, past_hi=0, mix=5),
        # one token of the small model: the latency of one call
        dict(name="cache8_tiny", op="decode8", **tiny, n=1, len_lo=256, len_hi=256, mix=6),
        # the benchmark's decode batch over an 8-bit cache
        dict(name="cache8_2p9b", op="decode8", **m29, n=16, len_lo=8192, len_hi=8192, mix=7),
        # a ragged serving batch
        dict(name="cache8_ragged", op="decode8", **m29, n=64, len_lo=1024, len_hi=32768, mix=8),
        # the MLA shape at 16k tokens a sequence
        dict(name="cache8_mla", op="decode8", **mla, n=32, len_lo=16384, len_hi=16384, mix=9),
        # the new token of each sequence of a decode step
        dict(name="append_step", op="append8", **m29, n=16, new_lo=1, new_hi=1, past_lo=500, past_hi=8191, mix=10),
        # accepted draft tokens of a speculative step, a few each
        dict(name="append_draft", op="append8", **mla2, n=64, new_lo=1, new_hi=7, past_lo=3, past_hi=2000, mix=11),
        # prompts of a batch written after their prefill
        dict(name="append_prompt", op="append8", **m29, n=12, new_lo=300, new_hi=8192, past_lo=0, past_hi=0, mix=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["prefill", "decode8", "append8"])
    shape = rng.choice([dict(branches=4, d_c=64, d_r=32), dict(branches=2, d_c=64, d_r=64), dict(branches=4, d_c=128, d_r=64),
                        dict(branches=4, d_c=128, d_r=64), dict(branches=1, d_c=128, d_r=64), dict(branches=2, d_c=256, d_r=64),
                        dict(branches=1, d_c=512, d_r=64), dict(branches=2, d_c=128, d_r=32), dict(branches=1, d_c=256, d_r=32)])
    c = dict(op=op, heads=rng.choice([1, 5, 8, 16, 16, 24, 40]), page=rng.choice([16, 32, 64, 64, 128]), mix=rng.randrange(1 << 20), **shape)
    most = {x["name"]: x for x in listed()}[{"prefill": "prompt_8k", "decode8": "cache8_ragged", "append8": "append_prompt"}[op]]
    while True:
        c["n"] = _log_int(rng, 1, 64 if op != "prefill" else 12)
        if op == "decode8":
            c["len_lo"], c["len_hi"] = sorted((_log_int(rng, 1, 32768), _log_int(rng, 1, 32768)))
        else:
            top = 8192 if op == "append8" else 4096
            c["new_lo"], c["new_hi"] = sorted((_log_int(rng, 1, top), _log_int(rng, 1, top)))
            c["past_lo"], c["past_hi"] = (0, 0) if rng.random() < 0.4 else sorted((rng.randrange(8000), rng.randrange(8000)))
        new, lens = _lens(c)
        w, top = work(c), work(most)
        padded = c["n"] * c["heads"] * c["branches"] * max(new) * max(lens)
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"] and (op != "prefill" or padded <= 64 * 8192 ** 2):
            return c


def _lens(c):
    """(new tokens, lengths with them) of the case's sequences."""
    rng = random.Random(c["mix"])
    if c["op"] == "decode8":
        return [1] * c["n"], [_log_int(rng, c["len_lo"], c["len_hi"]) for _ in range(c["n"])]
    new = [_log_int(rng, c["new_lo"], c["new_hi"]) for _ in range(c["n"])]
    return new, [q + rng.randint(c["past_lo"], c["past_hi"]) for q in new]


def work(c):
    new, lens = _lens(c)
    T, H, W, dr = sum(new), c["heads"], c["branches"] * c["d_c"], c["d_r"]
    scales = 4 * c["branches"] / BLOCK
    if c["op"] == "append8":
        return {"bytes": T * (2 * W + 2 * dr + W + 2 * dr + scales), "flops": T * (2 * W + 3 * dr)}
    rows = T * H * (4 * W + 2 * dr)  # queries in, outputs out
    if c["op"] == "decode8":
        return {"bytes": sum(lens) * (W + 2 * dr + scales) + rows, "flops": 2 * sum(lens) * H * (2 * W + dr)}
    pairs = sum(q * (n - q) + q * (q + 1) // 2 for q, n in zip(new, lens))
    return {"bytes": sum(lens) * 2 * (W + dr) + rows, "flops": 2 * pairs * H * (2 * W + dr)}


# ----------------------------------------------------------------- the inputs
def _power_scale(amax):
    """The smallest power of two s with amax <= 448 s, at least 2^-40."""
    m, e = torch.frexp(amax)
    return torch.ldexp(torch.ones_like(amax), (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=-40))


def prepare(c, seed):
    """Inputs of one call on the GPU: a paged pool in random page order, the
    sequences' tables and lengths, and the new tokens' rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, lens = _lens(c)
    N, H, B, dc, dr, P = c["n"], c["heads"], c["branches"], c["d_c"], c["d_r"], c["page"]
    T = sum(new)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)

    counts = [-(-n // P) for n in lens]
    pages, most = sum(counts) + 2, max(counts)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + counts[:-1], device="cuda").cumsum(0)
    at = torch.arange(most, device="cuda")
    used = at[None] < torch.tensor(counts, device="cuda")[:, None]
    table = torch.where(used, order[(first[:, None] + at[None]).clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
    s = dict(op=c["op"], block_table=table, seqlens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             cu_seqlens=torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32), max_new=max(new), max_len=max(lens),
             rope_cache=normal(pages, P, dr, std=dr ** -0.5), scale=(dc + dr) ** -0.5, out_scale=B ** -0.5)
    # latents of unit-norm rows whose size varies from token to token, as a
    # norm's gain and the tokens' own weight make it
    size = torch.exp(0.5 * torch.randn(pages, P, B, 1, generator=g, device="cuda"))
    latent = normal(pages, P, B, dc, std=dc ** -0.5) * size.to(torch.bfloat16)
    if c["op"] == "prefill":
        s["latent_cache"] = latent
    else:
        x = latent.float().view(pages, P // BLOCK, BLOCK, B, dc)
        scale = _power_scale(x.abs().amax((2, 4)))
        s["latent_scale"] = scale
        s["latent_cache"] = (x / scale[:, :, None, :, None]).to(torch.float8_e4m3fn).view(pages, P, B, dc)
    if c["op"] == "append8":
        size = torch.exp(0.5 * torch.randn(T, B, 1, generator=g, device="cuda"))
        s["c_new"] = normal(T, B, dc, std=dc ** -0.5) * size.to(torch.bfloat16)
        s["kr_new"] = normal(T, dr, std=dr ** -0.5)
        s["rope_base"] = 10000.0
    else:
        # scores of a standard deviation of about 2 at unit latents
        gain = 2.0 / (s["scale"] * math.sqrt(1.0 / dc + 1.0 / dr))
        s["q_lat"], s["q_rope"] = normal(T, H, B, dc, std=gain * dc ** -0.5), normal(T, H, dr, std=gain * dr ** -0.5)
    return s


# ----------------------------------------------------------------- one pass
def run(s):
    if own:
        from branch_latent_kv_b200 import mlra_append_fp8, mlra_decode_fp8, mlra_prefill
        if s["op"] == "prefill":
            return mlra_prefill(s["q_lat"], s["q_rope"], s["latent_cache"], s["rope_cache"], s["block_table"], s["seqlens"],
                                s["cu_seqlens"], s["scale"], s["out_scale"])
        if s["op"] == "decode8":
            return mlra_decode_fp8(s["q_lat"], s["q_rope"], s["latent_cache"], s["latent_scale"], s["rope_cache"], s["block_table"],
                                   s["seqlens"], s["scale"], s["out_scale"])
        mlra_append_fp8(s["c_new"], s["kr_new"], s["cu_seqlens"], s["seqlens"], s["block_table"], s["latent_cache"], s["latent_scale"],
                        s["rope_cache"], rope_base=s["rope_base"])
        return s["latent_cache"], s["latent_scale"], s["rope_cache"]
    return {"prefill": _prefill, "decode8": _decode8, "append8": _append8}[s["op"]](s)


def _rows(s, P):
    """Pool rows [N, max_len] of every sequence's tokens (row 0 past its end)."""
    t = torch.arange(s["max_len"], device="cuda")
    page = s["block_table"][:, t // P].long()
    return page.clamp(min=0) * P + t % P


def _softmax_(x):
    """exp(x - max) in place; its row sums beside it."""
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    return x.sum(-1, keepdim=True)


def _prefill(s):
    pages, P, B, dc = s["latent_cache"].shape
    T, H = s["q_lat"].shape[:2]
    rows = _rows(s, P)
    N, L, Q = rows.shape[0], s["max_len"], s["max_new"]
    lat = s["latent_cache"].view(pages * P, B, dc)[rows].float().permute(0, 2, 1, 3)  # [N, B, L, d_c]
    kr = s["rope_cache"].view(pages * P, -1)[rows].float()
    i = torch.arange(Q, device="cuda")
    start, stop = s["cu_seqlens"][:-1, None].long(), s["cu_seqlens"][1:, None].long()
    token = start + i  # [N, Q]
    real, at = token < stop, token.clamp(max=T - 1)
    pos = s["seqlens"][:, None].long() - (stop - start) + i
    q = s["q_lat"][at].float().permute(0, 3, 2, 1, 4).reshape(N, B, H * Q, dc)
    qr = s["q_rope"][at].float().permute(0, 2, 1, 3).reshape(N, 1, H * Q, -1)
    x = torch.matmul(q, lat.transpose(2, 3))
    x += torch.matmul(qr, kr[:, None].transpose(2, 3))
    x = x.mul_(s["scale"]).view(N, B, H, Q, L)
    x.masked_fill_((torch.arange(L, device="cuda") > pos[..., None])[:, None, None], float("-inf"))
    total = _softmax_(x)
    o = torch.matmul(x.view(N, B, H * Q, L), lat).view(N, B, H, Q, dc) / total * s["out_scale"]
    return o.permute(0, 3, 2, 1, 4)[real].to(torch.bfloat16)  # [T, H, B, d_c]


def _decode8(s):
    pages, P, B, dc = s["latent_cache"].shape
    rows = _rows(s, P)
    lat = s["latent_cache"].view(torch.uint8).view(pages * P, B, dc)[rows].view(torch.float8_e4m3fn).float()
    lat = (lat * s["latent_scale"].view(-1, B)[rows // BLOCK][..., None]).permute(0, 2, 1, 3)  # [N, B, L, d_c]
    kr = s["rope_cache"].view(pages * P, -1)[rows].float()
    x = torch.matmul(s["q_lat"].float().transpose(1, 2), lat.transpose(2, 3))  # [N, B, H, L]
    x += torch.matmul(s["q_rope"].float(), kr.transpose(1, 2))[:, None]
    past = torch.arange(s["max_len"], device="cuda") >= s["seqlens"][:, None]
    x.mul_(s["scale"]).masked_fill_(past[:, None, None], float("-inf"))
    total = _softmax_(x)
    return (torch.matmul(x, lat) / total * s["out_scale"]).transpose(1, 2).to(torch.bfloat16).contiguous()


def _append8(s):
    cache, scale, rope = s["latent_cache"], s["latent_scale"], s["rope_cache"]
    pages, P, B, dc = cache.shape
    T, dr = s["kr_new"].shape
    cu, L = s["cu_seqlens"].long(), s["seqlens"].long()
    i = torch.arange(T, device="cuda")
    n = torch.searchsorted(cu, i, right=True) - 1
    pos = L[n] - cu[n + 1] + i
    row = s["block_table"][n, pos // P].long() * P + pos % P  # the pool row of each new token
    # the scales: the largest finite new value of each block, and the block's
    # earlier scale where it holds tokens already
    x = s["c_new"].float()
    amax = torch.where(x.isfinite(), x.abs(), 0.0).amax(2)
    blocks = scale.view(-1, B)
    need = torch.full_like(blocks, -1.0).scatter_reduce_(0, (row // BLOCK)[:, None].expand(T, B), amax, "amax")
    old = blocks.clone()
    begin = L - (cu[1:] - cu[:-1])  # the first new position of each sequence
    held = (begin % BLOCK != 0) & (cu[1:] > cu[:-1])
    first = s["block_table"].gather(1, (begin // P).clamp(max=s["block_table"].shape[1] - 1)[:, None])[:, 0].long() * P + begin % P
    first = torch.where(held, first // BLOCK, blocks.shape[0])  # the block each sequence carries on
    carried = torch.zeros(blocks.shape[0] + 1, dtype=torch.bool, device="cuda").index_fill_(0, first, True)[:-1, None]
    fresh = _power_scale(need.clamp(min=0))
    blocks.copy_(torch.where(need >= 0, torch.where(carried, torch.maximum(old, fresh), fresh), old))
    # earlier rows of a carried block, rounded again at its new scale
    slot = torch.arange(BLOCK, device="cuda")
    again = (held[:, None] & (slot < (begin % BLOCK)[:, None])).nonzero()  # [(sequence, slot)]
    block = first[again[:, 0]]
    codes = cache.view(torch.uint8).view(-1, B, dc)
    at = block * BLOCK + again[:, 1]
    value = codes[at].view(torch.float8_e4m3fn).float() * (old[block] / blocks[block])[..., None]
    codes[at] = value.to(torch.float8_e4m3fn).view(torch.uint8)
    value = (x / blocks[row // BLOCK][..., None]).clamp(-TOP, TOP)
    codes[row] = value.to(torch.float8_e4m3fn).view(torch.uint8)
    # the RoPE keys: pair j turns by pos * base^(-2j/d_r), in 64 bits
    angle = pos.double()[:, None] * s["rope_base"] ** (torch.arange(0, dr, 2, device="cuda").double() * (-1.0 / dr))
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b = s["kr_new"].float().view(T, dr // 2, 2).unbind(-1)
    rope.view(-1, dr)[row] = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).view(T, dr).to(torch.bfloat16)
    return cache, scale, rope


# ----------------------------------------------------------------- in 64 bits
def exact(c, seed):
    s = prepare(c, seed)
    new, lens = _lens(c)
    P, B, H = c["page"], c["branches"], c["heads"]
    table, cache = s["block_table"].tolist(), s["latent_cache"].double()

    def gather(pool, n):  # sequence n's tokens in order
        return pool[torch.tensor(table[n][:-(-lens[n] // P)], device="cuda")].flatten(0, 1)[:lens[n]]

    if c["op"] == "append8":
        scale, rope = s["latent_scale"].double(), s["rope_cache"].double()
        done = 0
        for n, (q, length) in enumerate(zip(new, lens)):
            x, k = s["c_new"][done:done + q].double(), s["kr_new"][done:done + q].double()
            done += q
            begin = length - q
            for p0 in range(begin - begin % BLOCK, length, BLOCK):  # one block of 16 positions
                page, slot = table[n][p0 // P], p0 % P
                lo, hi = max(begin, p0), min(length, p0 + BLOCK)
                part = x[lo - begin:hi - begin]
                amax = part.abs().amax((0, 2)).clamp(min=TOP * 2.0 ** -40)
                fresh = torch.exp2(torch.ceil(torch.log2(amax / TOP)))  # a tie of log2 is exact at a power of two
                if lo > p0:
                    fresh = torch.maximum(fresh, scale[page, slot // BLOCK])
                    kept = cache[page, slot:slot + lo - p0] * (scale[page, slot // BLOCK] / fresh)[None, :, None]
                    cache[page, slot:slot + lo - p0] = kept.float().to(torch.float8_e4m3fn).double()
                scale[page, slot // BLOCK] = fresh
                cache[page, slot + lo - p0:slot + hi - p0] = (part / fresh[None, :, None]).float().to(torch.float8_e4m3fn).double()
            pos = torch.arange(begin, length, device="cuda")
            z = torch.view_as_complex(k.view(q, -1, 2))
            turn = torch.exp(-math.log(s["rope_base"]) * 2.0 / c["d_r"] * torch.arange(c["d_r"] // 2, device="cuda").double())
            z = z * torch.polar(torch.ones_like(z.real), pos.double()[:, None] * turn)
            page = torch.tensor(table[n], device="cuda")[pos // P]
            rope[page, pos % P] = torch.view_as_real(z).view(q, -1)
        return cache, scale, rope
    if c["op"] == "decode8":
        cache = cache * s["latent_scale"].double().repeat_interleave(BLOCK, 1)[..., None]
    out, done = torch.empty(s["q_lat"].shape, dtype=torch.float64, device="cuda"), 0
    for n, (q, length) in enumerate(zip(new, lens)):
        lat, kr = gather(cache, n), gather(s["rope_cache"].double(), n)
        later = torch.ones(q, length, dtype=torch.bool, device="cuda").triu(length - q + 1)
        for h in range(H):
            qr = s["q_rope"][done:done + q, h].double() @ kr.T
            for b in range(B):
                x = (s["q_lat"][done:done + q, h, b].double() @ lat[:, b].T + qr) * s["scale"]
                p = torch.softmax(x.masked_fill(later, -math.inf), 1)
                out[done:done + q, h, b] = p @ lat[:, b] * s["out_scale"]
        done += q
    return out
