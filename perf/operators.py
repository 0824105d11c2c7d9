"""Measured cases of the serving and training operators around the attention
calls: attention of a ragged chunk of new tokens over a paged cache
(``fwd_paged``), the append to that cache with the norm and the position
rotation on the way (``kvcache_append``), and the per-head norm with the
position rotation in one pass, forward and backward (``qk_norm_rope``,
``qk_norm_rope_bwd``).

``own`` chooses what ``run`` computes: False, the plain form in elementary
torch operations; True, the library's calls.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ----------------------------------------------------------------- the cases

def listed():
    """Twelve cases; each comment says what it stands for in real use."""
    return [
        # one token each for a few short conversations: launch latency counts
        _paged("paged_decode_8", batch=8, q_lo=1, q_hi=1, c_lo=1, c_hi=2048, page=16, hq=32,
               hkv=8, d=128, dtype="bf16", len_seed=11),
        # the decode step of a full server: 64 sequences, caches up to 32K, 256-token pages
        _paged("paged_decode_64", batch=64, q_lo=1, q_hi=1, c_lo=1, c_hi=32768, page=256, hq=32,
               hkv=8, d=128, dtype="bf16", len_seed=8),
        # a few drafted tokens checked per sequence, 64-wide heads, small pages
        _paged("paged_draft_d64", batch=24, q_lo=2, q_hi=9, c_lo=500, c_hi=16000, page=16, hq=64,
               hkv=8, d=64, dtype="fp16", len_seed=3),
        # a scheduler's mixed step: 47 single tokens and one prompt chunk of 2001 tokens
        _paged("paged_mixed_48", batch=48, q_lo=1, q_hi=1, q_last=2001, c_lo=1, c_hi=8192, page=64,
               hq=32, hkv=8, d=128, dtype="bf16", len_seed=5),
        # one long prompt's chunk of 8192 tokens behind 24576 cached ones
        _paged("paged_chunk_8192", batch=1, q_lo=8192, q_hi=8192, c_lo=24576, c_hi=24576, page=256,
               hq=32, hkv=8, d=128, dtype="bf16", len_seed=1),
        # ragged prompt chunks of a windowed, soft-capped layer with 256-wide heads
        _paged("paged_window_d256", batch=12, q_lo=100, q_hi=1000, c_lo=1, c_hi=4097, page=32,
               hq=8, hkv=4, d=256, dtype="bf16", len_seed=7, win_l=1024, softcap=50.0),
        # the same server's decode step before the attention: one token per sequence
        _append("append_decode_64", batch=64, q_lo=1, q_hi=1, c_lo=1, c_hi=1024, page=256, hq=32,
                hkv=8, d=128, dtype="bf16", len_seed=9, norm=True, rot=128, interleaved=False),
        # ragged prompt chunks entering small pages; no norm, interleaved pairs
        _append("append_prompt_16k", batch=12, q_lo=300, q_hi=2500, c_lo=0, c_hi=2048, page=16,
                hq=32, hkv=8, d=64, dtype="fp16", len_seed=4, norm=False, rot=64,
                interleaved=True),
        # the training shape's queries and keys
        _norm_rope("norm_rope_train", b=4, s=8192, hq=32, hkv=8, d=128, dtype="bf16", norm=True,
                   rot=128, interleaved=False, backward=False),
        # a short odd batch, half of each head rotated
        _norm_rope("norm_rope_odd_d64", b=3, s=331, hq=14, hkv=2, d=64, dtype="fp16", norm=True,
                   rot=32, interleaved=False, backward=False),
        # its gradient on the training shape
        _norm_rope("norm_rope_bwd_train", b=4, s=8192, hq=32, hkv=8, d=128, dtype="bf16",
                   norm=True, rot=128, interleaved=False, backward=True),
        # its gradient on the 256-wide sweep shape, odd length, interleaved pairs
        _norm_rope("norm_rope_bwd_d256", b=2, s=1023, hq=8, hkv=8, d=256, dtype="fp16", norm=True,
                   rot=256, interleaved=True, backward=True),
    ]


def _paged(name, *, batch, q_lo, q_hi, c_lo, c_hi, page, hq, hkv, d, dtype, len_seed, q_last=0,
           win_l=-1, softcap=0.0):
    return dict(name=name, op="paged", batch=batch, q_lo=q_lo, q_hi=q_hi, q_last=q_last, c_lo=c_lo,
                c_hi=c_hi, page=page, hq=hq, hkv=hkv, d=d, dtype=dtype, len_seed=len_seed,
                win_l=win_l, softcap=softcap)


def _append(name, *, batch, q_lo, q_hi, c_lo, c_hi, page, hq, hkv, d, dtype, len_seed, norm, rot,
            interleaved):
    return dict(name=name, op="append", batch=batch, q_lo=q_lo, q_hi=q_hi, q_last=0, c_lo=c_lo,
                c_hi=c_hi, page=page, hq=hq, hkv=hkv, d=d, dtype=dtype, len_seed=len_seed,
                norm=norm, rot=rot, interleaved=interleaved)


def _norm_rope(name, *, b, s, hq, hkv, d, dtype, norm, rot, interleaved, backward):
    return dict(name=name, op="norm_rope", b=b, s=s, hq=hq, hkv=hkv, d=d, dtype=dtype, norm=norm,
                rot=rot, interleaved=interleaved, backward=backward)


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ones' ranges: sizes over their logarithms."""
    kind = rng.choice(["decode", "chunk", "mixed", "append", "forward", "backward"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 5, 7, 8])
    dtype = rng.choice(["bf16", "fp16"])
    rot = rng.choice([d, d, d // 2])
    shape = dict(hq=hkv * g, hkv=hkv, d=d, dtype=dtype)
    norm, interleaved = rng.random() < 0.7, rng.random() < 0.4
    page = rng.choice([16, 32, 48, 64, 128, 256])
    seed = rng.randrange(1 << 30)
    window = rng.choice([-1, -1, _log_int(rng, 100, 4096)])
    cap = rng.choice([0.0, 0.0, 30.0])
    if kind == "decode":
        batch = _log_int(rng, 1, 64)
        q_hi = rng.choice([1, 1, 4, 9])
        return _paged("", batch=batch, q_lo=1, q_hi=q_hi, c_lo=1,
                      c_hi=_log_int(rng, 300, 32768), page=page, len_seed=seed, win_l=window,
                      softcap=cap, **shape)
    if kind == "chunk":
        batch = _log_int(rng, 1, 12)
        q_hi = max(2, _log_int(rng, 30, 8192) // batch)
        return _paged("", batch=batch, q_lo=max(1, q_hi // 3), q_hi=q_hi, c_lo=0,
                      c_hi=_log_int(rng, 100, 16384), page=page, len_seed=seed, win_l=window,
                      softcap=cap, **shape)
    if kind == "mixed":
        return _paged("", batch=_log_int(rng, 3, 64), q_lo=1, q_hi=1,
                      q_last=_log_int(rng, 50, 4000), c_lo=1, c_hi=_log_int(rng, 300, 16384),
                      page=page, len_seed=seed, win_l=window, softcap=cap, **shape)
    if kind == "append":
        batch = _log_int(rng, 1, 64)
        return _append("", batch=batch, q_lo=1, q_hi=max(1, _log_int(rng, 1, 16384) // batch),
                       c_lo=0, c_hi=_log_int(rng, 10, 2048), page=page, len_seed=seed, norm=norm,
                       rot=rot, interleaved=interleaved, **shape)
    rows = _log_int(rng, 64, 32768)
    b = rng.choice([1, 2, 3, 4])
    return _norm_rope("", b=b, s=max(1, rows // b), norm=norm, rot=rot, interleaved=interleaved,
                      backward=kind == "backward", **shape)


def _lengths(case):
    """(new tokens, cached tokens) of every sequence: part of the case, not of the seed."""
    rng = random.Random(case["len_seed"])
    new = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    if case["q_last"]:
        new[-1] = case["q_last"]
    cached = [rng.randint(case["c_lo"], case["c_hi"]) for _ in range(case["batch"])]
    return new, cached


def _visible(case):
    """(visible query-key pairs, keys that some query sees) over all sequences."""
    new, cached = _lengths(case)
    w = case["win_l"]
    pairs = keys = 0
    for n, c in zip(new, cached):
        first = 0 if w < 0 else max(0, c - w)
        keys += c + n - first
        if w < 0:
            pairs += n * c + n * (n + 1) // 2
        else:
            pairs += sum(min(c + i, w) + 1 for i in range(n))
    return pairs, keys


def work(case):
    """Bytes and operations that one pass cannot do without."""
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "paged":
        new, _ = _lengths(case)
        pairs, keys = _visible(case)
        rows = sum(new)
        # q and out, lse, the visible keys and values; two products per visible pair
        return {"bytes": 2 * rows * hq * d * 2 + 4 * rows * hq + 2 * keys * hkv * d * 2,
                "flops": 4 * pairs * hq * d}
    if case["op"] == "append":
        rows = sum(_lengths(case)[0])
        per = (6 if case["rot"] else 0) + (4 if case["norm"] else 0)
        # q, k, v in; q out and the cache rows out
        return {"bytes": 2 * rows * (hq + 2 * hkv) * d * 2,
                "flops": per * rows * (hq + hkv) * d}
    rows = case["b"] * case["s"]
    n = rows * (hq + hkv) * d
    if case["backward"]:
        # the inputs (the norm's gradient needs them), the gradients in and out
        return {"bytes": (3 if case["norm"] else 2) * n * 2, "flops": 14 * n}
    return {"bytes": 2 * n * 2, "flops": 8 * n}


# ---------------------------------------------------------------- the inputs

EPS = 1e-6
BASE = 10000.0


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    x = torch.empty(shape, device="cuda", dtype=dtype)
    x.normal_(0.0, scale, generator=g)
    return x


def _inv_freq(rot):
    j = torch.arange(rot // 2, dtype=torch.float64)
    return torch.pow(torch.tensor(BASE, dtype=torch.float64), -2.0 * j / max(rot, 1)).cuda()


def _i32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _pages(case, g, new, cached):
    """A block table of shuffled pages, one table row per sequence; entries past a
    sequence's last page are -1, as a page allocator leaves them."""
    page = case["page"]
    need = [-(-(c + n) // page) for c, n in zip(cached, new)]
    perm = torch.randperm(sum(need), generator=torch.Generator().manual_seed(g.initial_seed()))
    table = torch.full((len(need), max(need)), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n].to(torch.int32)
        at += n
    return table.cuda(), sum(need)


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    st = dict(case=case, scale=1.0 / math.sqrt(d))
    if case["op"] in ("paged", "append"):
        new, cached = _lengths(case)
        rows = sum(new)
        st["new"], st["cached"] = new, cached
        st["table"], pages = _pages(case, g, new, cached)
        st["pages"] = [-(-(c + n) // case["page"]) for c, n in zip(cached, new)]
        st["k_cache"] = _normal(g, (pages, case["page"], hkv, d), dt)
        st["v_cache"] = _normal(g, (pages, case["page"], hkv, d), dt)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        st["cu"], st["cu_dev"], st["cached_dev"] = cu, _i32(cu), _i32(cached)
        st["q"] = _normal(g, (rows, hq, d), dt)
    if case["op"] == "append":
        st["k_new"] = _normal(g, (rows, hkv, d), dt)
        st["v_new"] = _normal(g, (rows, hkv, d), dt)
        st["q_out"] = torch.empty_like(st["q"])
    if case["op"] == "norm_rope":
        b, s = case["b"], case["s"]
        st["q"] = _normal(g, (b, s, hq, d), dt)
        st["k"] = _normal(g, (b, s, hkv, d), dt)
        if case["backward"]:
            st["gq"] = _normal(g, (b, s, hq, d), dt, 0.02)
            st["gk"] = _normal(g, (b, s, hkv, d), dt, 0.02)
    if case["op"] != "paged":
        st["inv_freq"] = _inv_freq(case["rot"])
        st["wq"] = st["wk"] = None
        if case["norm"]:
            st["wq"] = 1.0 + _normal(g, (d,), torch.float32, 0.2)
            st["wk"] = 1.0 + _normal(g, (d,), torch.float32, 0.2)
            st["wq"], st["wk"] = st["wq"].to(dt), st["wk"].to(dt)
    if own:
        from exact_attention_41_gb300 import libattn

        if case["op"] == "paged":
            st["workspace"] = libattn.paged_workspace(st["q"], st["k_cache"], case["batch"])
        else:
            st["phases"] = libattn.rope_phases(st["inv_freq"])
            if case["op"] == "norm_rope" and case["backward"]:
                st["workspace"] = libattn.qk_norm_rope_bwd_workspace(st["q"], st["k"])
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    case = st["case"]
    if own:
        return _run_own(st, case)
    if case["op"] == "paged":
        return _plain_paged(st, case)
    if case["op"] == "append":
        return _plain_append(st, case)
    return _plain_norm_rope_bwd(st, case) if case["backward"] else _plain_norm_rope(st, case)


def _run_own(st, case):
    from exact_attention_41_gb300 import libattn

    if case["op"] == "paged":
        return libattn.fwd_paged(st["q"], st["k_cache"], st["v_cache"], st["cu_dev"],
                                 st["cached_dev"], block_table=st["table"], appended=True,
                                 causal=True, window=(case["win_l"], 0), softcap=case["softcap"],
                                 workspace=st["workspace"])
    rope = dict(phases=st["phases"], interleaved=case["interleaved"], q_weight=st["wq"],
                k_weight=st["wk"], eps=EPS)
    if case["op"] == "append":
        libattn.kvcache_append(st["k_new"], st["v_new"], st["k_cache"], st["v_cache"],
                               st["cu_dev"], st["cached_dev"], block_table=st["table"],
                               q=st["q"], q_out=st["q_out"], **rope)
        return st["q_out"], st["k_cache"], st["v_cache"]
    if case["backward"]:
        out = libattn.qk_norm_rope_bwd(st["q"], st["k"], st["gq"], st["gk"],
                                       workspace=st["workspace"], **rope)
        return [t for t in out if t is not None]
    return libattn.qk_norm_rope(st["q"], st["k"], **rope)


def _plain_paged(st, case):
    q, scale = st["q"], st["scale"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    g = hq // hkv
    out = torch.empty_like(q)
    lse = torch.empty((hq, q.shape[0]), device="cuda", dtype=torch.float32)
    cu = st["cu"]
    for i, (n, c) in enumerate(zip(st["new"], st["cached"])):
        keys = c + n
        first = 0 if case["win_l"] < 0 else max(0, c - case["win_l"])
        p0 = first // case["page"]
        idx = st["table"][i, p0:st["pages"][i]].long()
        lo, hi = first - p0 * case["page"], keys - p0 * case["page"]
        k = st["k_cache"][idx].reshape(-1, hkv, d)[lo:hi]
        v = st["v_cache"][idx].reshape(-1, hkv, d)[lo:hi]
        qi = q[cu[i]:cu[i + 1]]
        kf, vf = k.float().permute(1, 2, 0), v.float().transpose(0, 1)  # (hkv, d, L), (hkv, L, d)
        # query rows in pieces, so that the score matrix of a piece stays in memory
        step = max(1, (1 << 32) // (4 * hq * (keys - first)))
        key_at = torch.arange(first, keys, device="cuda")
        for r in range(0, n, step):
            m = min(step, n - r)
            qf = qi[r:r + m].float().reshape(m, hkv, g, d).transpose(0, 1).reshape(hkv, m * g, d)
            s = (qf @ kf) * scale
            if case["softcap"] > 0:
                s = torch.tanh(s / case["softcap"]) * case["softcap"]
            at = c + r + torch.arange(m, device="cuda").repeat_interleave(g)[:, None]
            dead = key_at[None, :] > at
            if case["win_l"] >= 0:
                dead = dead | (key_at[None, :] < at - case["win_l"])
            s = s.masked_fill(dead, float("-inf"))
            top = s.max(dim=2, keepdim=True).values
            p = torch.exp(s - top)
            total = p.sum(dim=2, keepdim=True)
            o = ((p @ vf) / total).reshape(hkv, m, g, d).transpose(0, 1)
            rows = slice(cu[i] + r, cu[i] + r + m)
            out[rows] = o.reshape(m, hq, d).to(q.dtype)
            z = (top + torch.log(total)).reshape(hkv, m, g)
            lse[:, rows] = z.transpose(1, 2).reshape(hq, m)
    return out, lse


def _angles(positions, inv_freq):
    """cos and sin of the rotation, in 64 bits because positions may be far, as 32-bit values."""
    a = positions.to(torch.float64)[:, None] * inv_freq[None, :]
    return torch.cos(a).float()[:, None, :], torch.sin(a).float()[:, None, :]


def _turn(x, cos, sin, rot, interleaved):
    """Rotates the first rot elements of the last dimension of x (rows, heads, d)."""
    if rot == 0:
        return x
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = a * sin + b * cos
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = a * sin + b * cos
    return y


def _norm_turn(x, w, cos, sin, case):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + EPS) * w.float()
    return _turn(y, cos, sin, case["rot"], case["interleaved"]).to(x.dtype)


def _plain_append(st, case):
    pos, row_page, row_slot = [], [], []
    for i, (n, c) in enumerate(zip(st["new"], st["cached"])):
        at = torch.arange(c, c + n, device="cuda")
        pos.append(at)
        row_page.append(st["table"][i].long()[at // case["page"]])
        row_slot.append(at % case["page"])
    pos, row_page, row_slot = torch.cat(pos), torch.cat(row_page), torch.cat(row_slot)
    cos, sin = _angles(pos, st["inv_freq"])
    st["q_out"].copy_(_norm_turn(st["q"], st["wq"], cos, sin, case))
    st["k_cache"][row_page, row_slot] = _norm_turn(st["k_new"], st["wk"], cos, sin, case)
    st["v_cache"][row_page, row_slot] = st["v_new"]
    return st["q_out"], st["k_cache"], st["v_cache"]


def _dense_angles(st, case):
    pos = torch.arange(case["s"], device="cuda").repeat(case["b"])
    return _angles(pos, st["inv_freq"])


def _plain_norm_rope(st, case):
    cos, sin = _dense_angles(st, case)
    return [_norm_turn(x.reshape(-1, x.shape[2], x.shape[3]), w, cos, sin, case).reshape(x.shape)
            for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"]))]


def _plain_norm_rope_bwd(st, case):
    cos, sin = _dense_angles(st, case)
    grads, weights = [], []
    for x, w, gy in ((st["q"], st["wq"], st["gq"]), (st["k"], st["wk"], st["gk"])):
        flat = (-1, x.shape[2], x.shape[3])
        gz = _turn(gy.reshape(flat).float(), cos, -sin, case["rot"], case["interleaved"])
        if w is not None:
            y = x.reshape(flat).float()
            r = torch.rsqrt((y * y).mean(dim=-1, keepdim=True) + EPS)
            y = y * r
            weights.append((gz * y).sum(dim=(0, 1), dtype=torch.float64).to(w.dtype))
            gz = gz * w.float()
            gz = (gz - y * (gz * y).mean(dim=-1, keepdim=True)) * r
        grads.append(gz.reshape(x.shape).to(x.dtype))
    return grads + weights


# ------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "paged":
        return _exact_paged(st, case)
    if case["op"] == "append":
        return _exact_append(st, case)
    return _exact_norm_rope(st, case)


def _exact_paged(st, case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    rows = st["q"].shape[0]
    out = torch.zeros((rows, hq, d), device="cuda", dtype=torch.float64)
    lse = torch.full((hq, rows), float("-inf"), device="cuda", dtype=torch.float64)
    base = 0
    for i in range(case["batch"]):
        n, c = st["new"][i], st["cached"][i]
        # token t of the sequence sits in page table[t / page], slot t % page
        t = torch.arange(c + n, device="cuda")
        page = st["table"][i].to(torch.int64)[torch.div(t, case["page"], rounding_mode="floor")]
        slot = torch.remainder(t, case["page"])
        for h in range(hq):
            kv = h * hkv // hq
            k = st["k_cache"][page, slot, kv].double()
            v = st["v_cache"][page, slot, kv].double()
            block = max(1, (1 << 27) // (c + n))
            for r in range(0, n, block):
                e = min(n, r + block)
                p = torch.arange(c + r, c + e, device="cuda").unsqueeze(1)
                x = torch.einsum("id,jd->ij", st["q"][base + r:base + e, h].double(), k) / d ** 0.5
                if case["softcap"] > 0:
                    x = case["softcap"] * torch.tanh(x / case["softcap"])
                seen = t.unsqueeze(0) <= p
                if case["win_l"] >= 0:
                    seen &= t.unsqueeze(0) >= p - case["win_l"]
                x = torch.where(seen, x, torch.full_like(x, float("-inf")))
                z = torch.logsumexp(x, dim=1)
                out[base + r:base + e, h] = torch.exp(x - z.unsqueeze(1)) @ v
                lse[h, base + r:base + e] = z
        base += n
    return out, lse


def _rotation(positions, case):
    """The rotation of every row as complex numbers exp(i pos f_j)."""
    j = torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float64)
    f = torch.exp(-(2.0 * j / max(case["rot"], 1)) * math.log(BASE))
    a = torch.outer(positions.double(), f)
    return torch.polar(torch.ones_like(a), a)


def _exact_map(x, w, z, case):
    """Norm and rotation of rows x (rows, heads, d), z the rows' rotation."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(torch.sum(y * y, dim=2, keepdim=True) / y.shape[2] + EPS) * w.double()
    rot = case["rot"]
    head, tail = y[:, :, :rot], y[:, :, rot:]
    if case["interleaved"]:
        c = torch.complex(head[:, :, 0::2].contiguous(), head[:, :, 1::2].contiguous())
    else:
        c = torch.complex(head[:, :, :rot // 2].contiguous(), head[:, :, rot // 2:].contiguous())
    c = c * z.unsqueeze(1)
    if case["interleaved"]:
        head = torch.stack((c.real, c.imag), dim=3).flatten(2)
    else:
        head = torch.cat((c.real, c.imag), dim=2)
    return torch.cat((head, tail), dim=2)


def _exact_append(st, case):
    pos = torch.cat([torch.arange(c, c + n) for n, c in zip(st["new"], st["cached"])]).cuda()
    z = _rotation(pos, case)
    q = _exact_map(st["q"], st["wq"], z, case)
    k = _exact_map(st["k_new"], st["wk"], z, case)
    k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
    flat_k, flat_v = k_cache.view(-1, *k.shape[1:]), v_cache.view(-1, *k.shape[1:])
    table = st["table"].cpu()
    at = 0
    for i, (n, c) in enumerate(zip(st["new"], st["cached"])):
        where = torch.tensor([int(table[i, t // case["page"]]) * case["page"] + t % case["page"]
                              for t in range(c, c + n)], device="cuda")
        flat_k[where] = k[at:at + n]
        flat_v[where] = st["v_new"][at:at + n].double()
        at += n
    return q, k_cache, v_cache


def _exact_norm_rope(st, case):
    z = _rotation(torch.arange(case["s"], device="cuda").repeat(case["b"]), case)
    grads, weights, outs = [], [], []
    for x, w, gy in ((st["q"], st["wq"], st.get("gq")), (st["k"], st["wk"], st.get("gk"))):
        rows = x.shape[0] * x.shape[1]
        flat = x.reshape(rows, x.shape[2], x.shape[3])
        if not case["backward"]:
            outs.append(_exact_map(flat, w, z, case).reshape(x.shape))
            continue
        # the gradient by automatic differentiation of the definition, in pieces of rows
        gx = torch.empty(flat.shape, device="cuda", dtype=torch.float64)
        gw = None if w is None else torch.zeros(x.shape[3], device="cuda", dtype=torch.float64)
        gflat = gy.reshape(flat.shape)
        for r in range(0, rows, 4096):
            leaf = flat[r:r + 4096].double().requires_grad_(True)
            wl = None if w is None else w.double().requires_grad_(True)
            with torch.enable_grad():
                y = _exact_map(leaf, wl, z[r:r + 4096], case)
                y.backward(gflat[r:r + 4096].double())
            gx[r:r + 4096] = leaf.grad
            if gw is not None:
                gw += wl.grad
        grads.append(gx.reshape(x.shape))
        if gw is not None:
            weights.append(gw)
    return grads + weights if case["backward"] else outs
