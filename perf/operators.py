"""Measured cases of the decode over shared prefixes, the cross attention and the cache-page operators.

Each case is one call (or the calls of one step) a program makes of this library:

  shared       fa.decode_shared: one token per sequence over a paged cache in which groups of sequences share
               their first pages (a system prompt, a document, the beams of one request)
  cross        fa.fwd_cross / fwd_varlen_cross: a decoder's prompt against an encoder's states of another length
  cross_train  the same forward and its backward
  cross_decode fa.decode_cross: one new token per sequence against its encoder states
  fork         fa.cache_fork: the beams of the next step, with copies of the partly filled pages
  append       fa.cache_append: new keys and values into the pages
  compact      fa.cache_collect and fa.cache_compact: the free list, then the used pages moved to the front

With ``own`` false, ``run`` computes the same in elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

PAGE = 16



# ------------------------------------------------------------------ cases

def listed():
    return [
        # a chat batch on a short system prompt: few sequences, little to read, latency counts
        {"name": "shared_small", "kind": "shared", "groups": "8", "prefix": "1000", "lo": 1, "hi": 64,
         "hq": 32, "hkv": 8, "d": 128},
        # a full decode batch on one system prompt of 4,096 tokens, answers of up to 1,024
        {"name": "shared_prompt", "kind": "shared", "groups": "64", "prefix": "4096", "lo": 16, "hi": 1024,
         "hq": 32, "hkv": 8, "d": 128},
        # questions about three long documents, 96 sequences in groups of unequal size
        {"name": "shared_documents", "kind": "shared", "groups": "48,31,17", "prefix": "24576,16391,30000",
         "lo": 256, "hi": 2048, "hq": 32, "hkv": 8, "d": 128},
        # several prompts sampled a few times each: small ragged groups, head dim 64, three heads to a KV head
        {"name": "shared_samples", "kind": "shared", "groups": "5,1,16,3,7,8", "prefix": "777,2048,4097,33,1500,0",
         "lo": 1, "hi": 700, "hq": 24, "hkv": 8, "d": 64},
        # a decoder's step over 64 utterances of up to 1,500 encoder states, no grouping of heads
        {"name": "cross_decode", "kind": "cross_decode", "b": 64, "nq": 1, "nk": 1500, "lo": 300, "hq": 16, "hkv": 16,
         "d": 64},
        # the decoder's prompt of the same model family at serving time: dense batch with padded encoder states
        {"name": "cross_prompt", "kind": "cross", "b": 16, "nq": 448, "nk": 1500, "lo": 400, "hq": 32, "hkv": 8,
         "d": 128},
        # training on packed pairs of ragged lengths, one of them without any encoder state
        {"name": "cross_train_packed", "kind": "cross_train", "b": 24, "packed": True, "nq": 1024, "qlo": 17, "nk": 2048,
         "lo": 1, "empty": 5, "hq": 16, "hkv": 16, "d": 64},
        # training on a dense batch with long encoder sequences: the largest products
        {"name": "cross_train_long", "kind": "cross_train", "b": 2, "packed": False, "nq": 2048, "nk": 8192, "lo": 8192,
         "hq": 32, "hkv": 8, "d": 128},
        # beam search over 16 requests of 4 beams: the winners of a step fork, partly filled pages are copied
        {"name": "fork_beams", "kind": "fork", "slots": 64, "beams": 4, "lo": 100, "hi": 4096, "hkv": 8, "d": 128},
        # one new token for each of 64 sequences: the smallest call
        {"name": "append_step", "kind": "append", "slots": 64, "old_lo": 100, "old_hi": 8192, "new_lo": 1, "new_hi": 1,
         "hkv": 8, "d": 128},
        # the keys and values of sixteen prompts after their prefill
        {"name": "append_prompts", "kind": "append", "slots": 16, "old_lo": 0, "old_hi": 500, "new_lo": 256,
         "new_hi": 8192, "hkv": 8, "d": 128},
        # a cache of 8,192 pages after many sequences have left: the rest moves to the front
        {"name": "compact_half", "kind": "compact", "slots": 48, "lo": 200, "hi": 3000, "pages": 8192, "hkv": 8,
         "d": 128},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    hq, hkv, d = rng.choice([(32, 8, 128), (16, 16, 64), (24, 8, 64), (20, 4, 128), (8, 1, 128), (8, 8, 128), (14, 2, 64)])
    kind = rng.choice(["shared", "shared", "shared", "cross", "cross_train", "cross_train", "cross_decode", "fork", "append",
                       "compact"])
    if kind == "shared":
        groups = [_log_int(rng, 1, 40) for _ in range(_log_int(rng, 1, 6))]
        while sum(groups) > 90:
            groups.pop()
        return {"kind": kind, "groups": ",".join(map(str, groups)),
                "prefix": ",".join(str(_log_int(rng, 1, 24000)) for _ in groups), "lo": 1, "hi": _log_int(rng, 1, 2000),
                "hq": hq, "hkv": hkv, "d": d}
    if kind == "cross_decode":
        return {"kind": kind, "b": _log_int(rng, 1, 64), "nq": rng.choice([1, 1, 1, 2, 5]), "nk": _log_int(rng, 3, 8000),
                "lo": 1, "hq": hq, "hkv": hkv, "d": d}
    if kind in ("cross", "cross_train"):
        b = _log_int(rng, 1, 12)
        nq, nk = _log_int(rng, 1, 1500), _log_int(rng, 1, 4000)
        packed = kind == "cross_train" and rng.random() < 0.5
        case = {"kind": kind, "b": b, "nq": nq, "nk": nk, "lo": rng.randint(1, nk), "hq": hq, "hkv": hkv, "d": d}
        if kind == "cross_train":
            case["packed"] = packed
        if packed:
            case["qlo"] = rng.randint(1, nq)
        return case
    if kind == "fork":
        beams = rng.choice([2, 3, 4, 8])
        return {"kind": kind, "slots": beams * _log_int(rng, 1, 24), "beams": beams, "lo": 1, "hi": _log_int(rng, 1, 6000),
                "hkv": hkv, "d": d}
    if kind == "append":
        new_hi = rng.choice([1, 1, _log_int(rng, 1, 5000)])
        return {"kind": kind, "slots": _log_int(rng, 1, 32), "old_lo": 0, "old_hi": _log_int(rng, 1, 8000), "new_lo": 1,
                "new_hi": new_hi, "hkv": hkv, "d": d}
    return {"kind": kind, "slots": _log_int(rng, 1, 64), "lo": 1, "hi": _log_int(rng, 1, 2500),
            "pages": rng.randint(7000, 11000), "hkv": hkv, "d": d}


def _ints(text):
    return [int(x) for x in text.split(",")]


def _spread(case, n, lo, hi, salt):
    """n lengths over [lo, hi], fixed by the case."""
    r = random.Random("%s %d %d %d %d" % (case["kind"], n, lo, hi, salt))
    return [r.randint(lo, hi) for _ in range(n)]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _shared_lens(case):
    groups, prefix = _ints(case["groups"]), _ints(case["prefix"])
    tails = _spread(case, sum(groups), case["lo"], case["hi"], 1)
    lens, s = [], 0
    for g, p in zip(groups, prefix):
        for _ in range(g):
            lens.append(p + tails[s])
            s += 1
    return groups, prefix, lens


def _cross_lens(case):
    nk = _spread(case, case["b"], case["lo"], case["nk"], 2)
    if case.get("empty") is not None:
        nk[case["empty"]] = 0
    if case.get("packed"):
        nq = _spread(case, case["b"], case["qlo"], case["nq"], 3)
    else:
        nq = [case["nq"]] * case["b"]
    return nq, nk


def _fork_lens(case):
    lens = _spread(case, case["slots"], case["lo"], case["hi"], 4)
    r = random.Random("parents %d %d" % (case["slots"], case["beams"]))
    parents = []
    for i in range(case["slots"]):     # a beam's parent is one of its request's beams
        base = i - i % case["beams"]
        parents.append(base + r.randrange(case["beams"]))
    return lens, parents


def work(case):
    d, hkv = case["d"], case["hkv"]
    kind = case["kind"]
    row = 4 * hkv * d                      # one token's K and V, bf16
    if kind == "shared":
        groups, prefix, lens = _shared_lens(case)
        full = [p // PAGE * PAGE for p in prefix]
        per_seq = [f for f, g in zip(full, groups) for _ in range(g)]
        keys = sum(full) + sum(n - f for n, f in zip(lens, per_seq))
        s = len(lens)
        return {"bytes": keys * row + s * case["hq"] * (4 * d + 4) + 4 * sum(_pages(n) for n in lens),
                "flops": 4 * case["hq"] * d * sum(lens)}
    if kind in ("cross", "cross_train", "cross_decode"):
        nq, nk = _cross_lens(case)
        pairs = sum(a * b for a, b in zip(nq, nk))
        q_bytes, kv_bytes = 2 * sum(nq) * case["hq"] * d, sum(nk) * row
        flops = 4 * case["hq"] * d * pairs
        total = 2 * q_bytes + kv_bytes + 4 * sum(nq) * case["hq"]
        if kind == "cross_train":          # q, o, do, k, v, lse in; dq, dk, dv out
            stored = sum(nk) if case.get("packed") else case["b"] * case["nk"]
            total += 4 * q_bytes + kv_bytes + 4 * sum(nq) * case["hq"] + stored * row
            flops += 10 * case["hq"] * d * pairs
        return {"bytes": total, "flops": flops}
    if kind == "fork":
        lens, parents = _fork_lens(case)
        moved = sum(lens[p] % PAGE for i, p in enumerate(parents) if p in parents[:i])
        return {"bytes": 2 * moved * row + 8 * sum(_pages(lens[p]) for p in parents), "flops": 0}
    if kind == "append":
        new = _spread(case, case["slots"], case["new_lo"], case["new_hi"], 6)
        return {"bytes": 2 * sum(new) * row, "flops": 0}
    lens, tables, live = _compact_tables(case)
    n_live = len(live)
    moved = sum(p >= n_live for p in live)
    return {"bytes": 2 * moved * PAGE * row + 8 * sum(_pages(n) for n in lens) + 4 * (case["pages"] - n_live), "flops": 0}


def _compact_tables(case):
    lens = _spread(case, case["slots"], case["lo"], case["hi"], 7)
    r = random.Random("pages %d %d" % (case["pages"], case["slots"]))
    while sum(_pages(n) for n in lens) > case["pages"] * 3 // 4:
        lens = [max(1, n // 2) for n in lens]
    order = r.sample(range(case["pages"]), sum(_pages(n) for n in lens))
    tables, at = [], 0
    for n in lens:
        tables.append(order[at:at + _pages(n)])
        at += _pages(n)
    return lens, tables, order


# ----------------------------------------------------------------- inputs

def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _table(rows, width):
    return _i32([list(r) + [-1] * (width - len(r)) for r in rows])


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rng = random.Random(seed)
    kind, d, hkv = case["kind"], case["d"], case["hkv"]
    st = {"kind": kind, "case": case}
    if kind == "shared":
        groups, prefix, lens = _shared_lens(case)
        full = [p // PAGE for p in prefix]
        total = sum(full) + sum(_pages(n) for n in lens) - sum(f * g for f, g in zip(full, groups))
        order = list(range(total))
        rng.shuffle(order)
        at, rows, s = 0, [], 0
        for g, f in zip(groups, full):
            first = order[at:at + f]
            at += f
            for _ in range(g):
                n = _pages(lens[s]) - f
                rows.append(first + order[at:at + n])
                at += n
                s += 1
        width = max(len(r) for r in rows)
        st.update(q=_randn((len(lens), case["hq"], d), gen), k=_randn((total, PAGE, hkv, d), gen),
                  v=_randn((total, PAGE, hkv, d), gen), table=_table(rows, width), lens=_i32(lens),
                  cu=_i32(_cu(groups)), prefix=_i32(prefix))
        return st
    if kind in ("cross", "cross_train", "cross_decode"):
        nq, nk = _cross_lens(case)
        if case.get("packed"):
            tq, tk = sum(nq), sum(nk)
            st.update(q=_randn((tq, case["hq"], d), gen), k=_randn((tk, hkv, d), gen), v=_randn((tk, hkv, d), gen),
                      cu_q=_i32(_cu(nq)), cu_k=_i32(_cu(nk)), max_q=max(nq), max_k=max(nk))
        else:
            b = case["b"]
            st.update(q=_randn((b, case["nq"], case["hq"], d), gen), k=_randn((b, case["nk"], hkv, d), gen),
                      v=_randn((b, case["nk"], hkv, d), gen), lens=_i32(nk))
        if kind == "cross_train":
            st["do"] = _randn(tuple(st["q"].shape), gen)
        return st
    if kind == "compact":
        lens, tables, _ = _compact_tables(case)
        total = case["pages"]
    else:
        if kind == "fork":
            lens, parents = _fork_lens(case)
            extra = case["slots"]
            st["parents"] = _i32(parents)
        else:
            lens = _spread(case, case["slots"], case["old_lo"], case["old_hi"], 5)
            new = _spread(case, case["slots"], case["new_lo"], case["new_hi"], 6)
            extra = sum(_pages(a + b) - _pages(a) for a, b in zip(lens, new))
            st["cu_new"] = _i32(_cu(new))
            st["k_new"] = _randn((sum(new), hkv, d), gen)
            st["v_new"] = _randn((sum(new), hkv, d), gen)
        total = sum(_pages(n) for n in lens) + extra + 7
        order = list(range(total))
        rng.shuffle(order)
        tables, at = [], 0
        for n in lens:
            tables.append(order[at:at + _pages(n)])
            at += _pages(n)
        free = sorted(order[at:], reverse=True)
        st["free"], st["count"] = _i32(free), _i32([len(free)])
        st["count_out"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    width = max(_pages(n) for n in lens) + 1
    if kind == "append":
        width = max(_pages(a + b) for a, b in zip(lens, new))
    st.update(k=_randn((total, PAGE, hkv, d), gen), v=_randn((total, PAGE, hkv, d), gen), lens=_i32(lens),
              table=_table(tables, width))
    st["lens_out"] = torch.zeros_like(st["lens"])
    if kind in ("fork", "compact"):
        st["table_out"] = torch.full_like(st["table"], -1)
    if kind == "compact":
        st["free"] = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        st["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        st["free_out"] = torch.full((total,), -1, dtype=torch.int32, device="cuda")
        st["count_out"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return st


# ------------------------------------------------------------- plain forms

def _softmax_av(q, k, v, seen, scale):
    """q [B,I,H,G,D], k, v [B,J,H,D] in 32 bits, seen [B,J] -> O [B,I,H,G,D], LSE [B,H,G,I], P [B,H,G,I,J]."""
    v = v.masked_fill(~seen[:, :, None, None], 0.0)
    k = k.masked_fill(~seen[:, :, None, None], 0.0)
    s = torch.einsum("bihgd,bjhd->bhgij", q, k) * scale
    s = s.masked_fill(~seen[:, None, None, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    o = torch.einsum("bhgij,bjhd->bihgd", p, v)
    return o, (torch.log(total) + m)[..., 0], p, k, v


def _split_heads(q, hkv):
    b, i, hq, d = q.shape
    return q.float().view(b, i, hkv, hq // hkv, d)


def _plain_shared(st):
    # every sequence's keys through its own row of the block table: the definition, without the sharing
    q, table, lens = st["q"], st["table"].long().clamp(min=0), st["lens"]
    s, hq, d = q.shape
    hkv = st["k"].shape[2]
    j = table.shape[1] * PAGE
    k = st["k"][table].view(s, j, hkv, d).float()
    v = st["v"][table].view(s, j, hkv, d).float()
    seen = torch.arange(j, device=q.device)[None, :] < lens[:, None]
    o, lse, _, _, _ = _softmax_av(_split_heads(q[:, None], hkv), k, v, seen, 1.0 / math.sqrt(d))
    return {"o": o.reshape(s, hq, d).to(torch.bfloat16), "lse": lse.reshape(s, hq)}


def _plain_cross_dense(q, k, v, do, seen):
    b, i, hq, d = q.shape
    hkv = k.shape[2]
    scale = 1.0 / math.sqrt(d)
    qs = _split_heads(q, hkv)
    o, lse, p, kf, vf = _softmax_av(qs, k.float(), v.float(), seen, scale)
    out = {"o": o.reshape(b, i, hq, d), "lse": lse.reshape(b, hq, i)}
    if do is not None:
        g = _split_heads(do, hkv)
        row = (g * o).sum(-1).permute(0, 2, 3, 1)[..., None]
        ds = p * (torch.einsum("bihgd,bjhd->bhgij", g, vf) - row) * scale
        out["dq"] = torch.einsum("bhgij,bjhd->bihgd", ds, kf).reshape(b, i, hq, d)
        out["dk"] = torch.einsum("bhgij,bihgd->bjhd", ds, qs)
        out["dv"] = torch.einsum("bhgij,bihgd->bjhd", p, g)
    return out


def _pad(x, cu, most):
    pos = torch.arange(most, device=x.device)[None, :]
    ok = pos < (cu[1:] - cu[:-1])[:, None]
    at = (cu[:-1, None] + pos).clamp(max=max(x.shape[0] - 1, 0)).long()
    return x[at].masked_fill(~ok[:, :, None, None], 0.0), ok


def _unpad(x, cu, total):
    t = torch.arange(total, device=x.device)
    s = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return x[s, t - cu.long()[s]]


def _plain_cross(st):
    q, k, v, do = st["q"], st["k"], st["v"], st.get("do")
    if "cu_q" in st:
        cu_q, cu_k, tq, tk = st["cu_q"], st["cu_k"], q.shape[0], k.shape[0]
        kp, seen = _pad(k, cu_k, st["max_k"])
        out = _plain_cross_dense(_pad(q, cu_q, st["max_q"])[0], kp, _pad(v, cu_k, st["max_k"])[0],
                                 None if do is None else _pad(do, cu_q, st["max_q"])[0], seen)
        out = {n: _unpad(x.transpose(1, 2), cu_q, tq).t().contiguous() if n == "lse"
               else _unpad(x, cu_k if n in ("dk", "dv") else cu_q, tk if n in ("dk", "dv") else tq)
               for n, x in out.items()}
    else:
        seen = torch.arange(k.shape[1], device=q.device)[None, :] < st["lens"][:, None]
        out = _plain_cross_dense(q, k, v, do, seen)
    return {n: x if n == "lse" else x.to(torch.bfloat16) for n, x in out.items()}


def _used(lens):
    return (lens.long() + PAGE - 1) // PAGE


def _plain_fork(st):
    table, lens, parents = st["table"], st["lens"].long(), st["parents"].long()
    n, width = parents.numel(), table.shape[1]
    here = torch.arange(n, device=table.device)
    first = torch.full((table.shape[0],), n, device=table.device).scatter_reduce(0, parents, here, "amin")
    length = lens[parents]
    copies = (length % PAGE > 0) & (first[parents] != here)
    order = torch.cumsum(copies.long(), 0) - 1
    rows, used = table[parents], _used(length)
    last = rows.gather(1, (used - 1).clamp(min=0)[:, None])[:, 0].long()
    fresh = st["free"][(st["count"].long() - 1 - order).clamp(min=0, max=st["free"].numel() - 1)].long()
    target = torch.where(copies, fresh, last)
    cols = torch.arange(width, device=table.device)[None, :]
    rows = torch.where((cols == (used - 1)[:, None]) & copies[:, None], target[:, None].int(), rows)
    st["table_out"].copy_(torch.where(cols < used[:, None], rows, st["table_out"]))
    tok = torch.arange(PAGE, device=table.device)[None, :]
    keep = tok < (length % PAGE)[:, None]
    src = (last[:, None] * PAGE + tok).reshape(-1)
    dst = torch.where(keep, target[:, None] * PAGE + tok, last[:, None] * PAGE + tok).reshape(-1)
    for_rows = (-1,) + tuple(st["k"].shape[2:])
    st["k"].view(for_rows).index_copy_(0, dst, st["k"].view(for_rows)[src])
    st["v"].view(for_rows).index_copy_(0, dst, st["v"].view(for_rows)[src])
    st["lens_out"].copy_(length)
    st["count_out"].copy_(st["count"] - copies.sum())
    return _fork_out(st)


def _fork_out(st):
    return {"table": st["table_out"], "lens": st["lens_out"], "count": st["count_out"], "k": st["k"], "v": st["v"]}


def _plain_append(st):
    table, lens, cu = st["table"], st["lens"].long(), st["cu_new"].long()
    new = cu[1:] - cu[:-1]
    used, used_new = _used(lens), _used(lens + new)
    before = torch.cumsum(used_new - used, 0) - (used_new - used)
    cols = torch.arange(table.shape[1], device=table.device)[None, :]
    taken = (st["count"].long() - 1 - (before[:, None] + cols - used[:, None])).clamp(min=0, max=st["free"].numel() - 1)
    fresh = (cols >= used[:, None]) & (cols < used_new[:, None])
    table.copy_(torch.where(fresh, st["free"][taken], table))
    t = torch.arange(st["k_new"].shape[0], device=table.device)
    s = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    pos = lens[s] + t - cu[s]
    at = table[s, pos // PAGE].long() * PAGE + pos % PAGE
    for_rows = (-1,) + tuple(st["k"].shape[2:])
    st["k"].view(for_rows).index_copy_(0, at, st["k_new"])
    st["v"].view(for_rows).index_copy_(0, at, st["v_new"])
    st["lens_out"].copy_(lens + new)
    st["count_out"].copy_(st["count"] - (used_new - used).sum())
    return _append_out(st)


def _append_out(st):
    return {"table": st["table"], "lens": st["lens_out"], "count": st["count_out"], "k": st["k"], "v": st["v"]}


def _plain_in_use(table, lens, pages):
    cols = torch.arange(table.shape[1], device=table.device)[None, :]
    named = torch.where(cols < _used(lens)[:, None], table.long(), pages).reshape(-1)
    return torch.zeros(pages + 1, dtype=torch.bool, device=table.device).index_fill_(0, named, True)[:pages]


def _plain_free_list(in_use, out, count):
    pages = in_use.numel()
    free = (~in_use).flip(0)
    where = torch.where(free, torch.cumsum(free.long(), 0) - 1, pages)
    ids = torch.arange(pages - 1, -1, -1, device=in_use.device, dtype=torch.int32)
    buf = torch.cat([out, out[:1]]).index_copy_(0, where, ids)[:pages]
    out.copy_(buf)
    count.copy_(free.sum()[None])


def _plain_compact(st):
    pages = st["k"].shape[0]
    in_use = _plain_in_use(st["table"], st["lens"], pages)
    _plain_free_list(in_use, st["free"], st["count"])
    ids = torch.arange(pages, device=in_use.device)
    live = in_use.sum()
    hole, mover = ~in_use & (ids < live), in_use & (ids >= live)
    # the i-th mover goes to the i-th hole: by rank, through a table of the holes
    rank_h = torch.where(hole, torch.cumsum(hole.long(), 0) - 1, pages)
    holes = torch.zeros(pages + 1, dtype=torch.long, device=ids.device).index_copy_(0, rank_h, ids)
    rank_m = torch.where(mover, torch.cumsum(mover.long(), 0) - 1, pages)
    to = torch.where(mover, holes[rank_m], ids)
    movers = torch.zeros(pages + 1, dtype=torch.long, device=ids.device).index_copy_(0, rank_m, ids)
    source = torch.where(hole, movers[rank_h], ids)
    st["k"].copy_(st["k"][source])
    st["v"].copy_(st["v"][source])
    cols = torch.arange(st["table"].shape[1], device=ids.device)[None, :]
    renamed = to[st["table"].long().clamp(min=0)].int()
    st["table_out"].copy_(torch.where(cols < _used(st["lens"])[:, None], renamed, st["table_out"]))
    _plain_free_list(ids < live, st["free_out"], st["count_out"])
    return _compact_out(st)


def _compact_out(st):
    return {"free": st["free"], "count": st["count"], "table": st["table_out"], "free_out": st["free_out"],
            "count_out": st["count_out"], "k": st["k"], "v": st["v"]}


# -------------------------------------------------------------------- run

def _own(st):
    import exact_io_aware_75_b200 as fa
    kind = st["kind"]
    if kind == "shared":
        o, lse = fa.decode_shared(st["q"], st["k"], st["v"], st["table"], st["lens"], st["cu"], st["prefix"])
        return {"o": o, "lse": lse}
    if kind == "cross_decode":
        o, lse = fa.decode_cross(st["q"], st["k"], st["v"], st["lens"])
        return {"o": o, "lse": lse}
    if kind in ("cross", "cross_train"):
        if "cu_q" in st:
            o, lse = fa.fwd_varlen_cross(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], st["max_q"], st["max_k"])
        else:
            o, lse = fa.fwd_cross(st["q"], st["k"], st["v"], st["lens"])
        out = {"o": o, "lse": lse}
        if kind == "cross_train":
            if "cu_q" in st:
                grads = fa.bwd_varlen_cross(st["q"], st["k"], st["v"], o, st["do"], lse, st["cu_q"], st["cu_k"],
                                            st["max_q"], st["max_k"])
            else:
                grads = fa.bwd_cross(st["q"], st["k"], st["v"], o, st["do"], lse, st["lens"])
            out.update(zip(("dq", "dk", "dv"), grads))
        return out
    if kind == "fork":
        fa.cache_fork(st["k"], st["v"], st["table"], st["lens"], st["parents"], st["free"], st["count"],
                      st["table_out"], st["lens_out"], st["count_out"])
        return _fork_out(st)
    if kind == "append":
        fa.cache_append(st["k_new"], st["v_new"], st["cu_new"], st["k"], st["v"], st["table"], st["lens"], st["free"],
                        st["count"], st["lens_out"], st["count_out"])
        return _append_out(st)
    fa.cache_collect(st["table"], st["lens"], st["free"], st["count"])
    fa.cache_compact(st["k"], st["v"], st["table"], st["lens"], st["table_out"], st["free_out"], st["count_out"])
    return _compact_out(st)


def run(state):
    if own:
        return _own(state)
    kind = state["kind"]
    if kind == "shared":
        return _plain_shared(state)
    if kind in ("cross", "cross_train", "cross_decode"):
        return _plain_cross(state)
    return {"fork": _plain_fork, "append": _plain_append, "compact": _plain_compact}[kind](state)


# ------------------------------------------------------------------ exact

def exact(case, seed):
    """The definition in 64 bits, one sequence and one query head at a time.  The cache operators move values and
    compute none."""
    if case["kind"] in ("fork", "append", "compact"):
        return None
    st = prepare(case, seed)
    q, k, v, do = st["q"], st["k"], st["v"], st.get("do")
    d, g = case["d"], case["hq"] // case["hkv"]
    if case["kind"] == "shared":
        _, _, lens = _shared_lens(case)
        o, lse = torch.zeros(q.shape, dtype=torch.float64, device=q.device), torch.zeros(q.shape[:2], dtype=torch.float64,
                                                                                          device=q.device)
        for s, n in enumerate(lens):
            pages = st["table"][s, :_pages(n)].long()
            keys = k[pages].flatten(0, 1)[:n].double().repeat_interleave(g, 1)
            vals = v[pages].flatten(0, 1)[:n].double().repeat_interleave(g, 1)
            x = (keys * q[s].double()[None]).sum(-1) * d ** -0.5              # [n, hq]
            lse[s] = torch.logsumexp(x, 0)
            o[s] = (torch.softmax(x, 0)[:, :, None] * vals).sum(0)
        return {"o": o, "lse": lse}
    nq, nk = _cross_lens(case)
    packed = bool(case.get("packed"))
    names = ("q", "k", "v") + (("do",) if do is not None else ())
    out = {"o": torch.zeros(q.shape, dtype=torch.float64, device=q.device),
           "lse": torch.full((case["hq"], sum(nq)) if packed else (case["b"], case["hq"], case["nq"]), -math.inf,
                             dtype=torch.float64, device=q.device)}
    if do is not None:
        for name in ("q", "k", "v"):
            out["d" + name] = torch.zeros(st[name].shape, dtype=torch.float64, device=q.device)
    a = c = 0
    for b in range(case["b"]):
        where = {n: (slice(a, a + nq[b]) if n in ("q", "do", "o", "dq") else slice(c, c + nk[b])) if packed
                 else (b, slice(0, nq[b] if n in ("q", "do", "o", "dq") else nk[b]))
                 for n in ("q", "k", "v", "do", "o", "dq", "dk", "dv")}
        a, c = a + nq[b], c + nk[b]
        if not nk[b]:
            continue
        part = {n: st[n][where[n]].double() for n in names}
        for h in range(case["hq"]):
            qh, kh, vh = part["q"][:, h], part["k"][:, h // g], part["v"][:, h // g]
            x = (qh @ kh.t()) * d ** -0.5
            w = torch.softmax(x, 1)
            oh = w @ vh
            out["o"][where["o"]][:, h] = oh
            if packed:
                out["lse"][h, a - nq[b]:a] = torch.logsumexp(x, 1)
            else:
                out["lse"][b, h] = torch.logsumexp(x, 1)
            if do is not None:
                gh = part["do"][:, h]
                dx = w * (gh @ vh.t() - (gh * oh).sum(1, keepdim=True)) * d ** -0.5
                out["dq"][where["dq"]][:, h] = dx @ kh
                out["dk"][where["dk"]][:, h // g] += dx.t() @ qh
                out["dv"][where["dv"]][:, h // g] += w.t() @ gh
    return out
