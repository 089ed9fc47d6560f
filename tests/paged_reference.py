"""Plain 64-bit definitions of the serving operators, for their tests: loops
over lists, on the CPU, sharing nothing with the library."""
from __future__ import annotations

import math

import torch


def attention(q, k_pool, v_pool, tables, lengths, scale):
    """(out, lse) in binary64; positions without a valid page are left out."""
    q, k_pool, v_pool = (t.detach().cpu().double() for t in (q, k_pool, v_pool))
    pages, ps, kv, d = k_pool.shape
    group = q.shape[1] // kv
    out = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    bound = torch.zeros(q.shape[:2], dtype=torch.float64)  # max_p sum_d |q k| scale
    for b, (row, n) in enumerate(zip(tables.tolist(), lengths.tolist())):
        at = [(row[p // ps], p % ps) for p in range(min(max(n, 0), len(row) * ps))]
        at = [(g, s) for g, s in at if 0 <= g < pages]
        if not at:
            continue
        g, s = (torch.tensor(x) for x in zip(*at))
        for h in range(q.shape[1]):
            k, v = k_pool[g, s, h // group], v_pool[g, s, h // group]
            x = (k @ q[b, h]) * scale
            lse[b, h] = torch.logsumexp(x, 0)
            out[b, h] = torch.exp(x - lse[b, h]) @ v
            bound[b, h] = (k.abs() @ q[b, h].abs()).max() * abs(scale)
    return out, lse, bound


def free(refs, tables, lengths, rows):
    refs, tables, lengths = list(refs), [list(r) for r in tables], list(lengths)
    for r in rows:
        if 0 <= r < len(tables):
            for p in tables[r]:
                if 0 <= p < len(refs):
                    refs[p] -= 1
            tables[r], lengths[r] = [-1] * len(tables[r]), 0
    return refs, tables, lengths


def extend(refs, tables, lengths, rows, counts, ps):
    refs, tables, lengths = list(refs), [list(r) for r in tables], list(lengths)
    free_pages = [p for p, n in enumerate(refs) if n <= 0]
    seen, wanted, done = set(), 0, []
    for r, c in zip(rows, counts):
        good = 0 <= r < len(tables) and r not in seen and c >= 0
        seen.add(r)
        good = good and max(lengths[r], 0) + c <= len(tables[r]) * ps
        if not good:
            done.append(0)
            continue
        n = max(lengths[r], 0)
        had, has = -(-n // ps), -(-(n + c) // ps)
        first, wanted = wanted, wanted + has - had
        done.append(int(wanted <= len(free_pages)))
        if done[-1]:
            for j in range(had, has):
                p = free_pages[first + j - had]
                tables[r][j], refs[p] = p, 1
            lengths[r] = n + c
    return refs, tables, lengths, done


def fork(refs, tables, lengths, parents, children, ps):
    """(refs, tables, lengths, done, copies): copies are (source, target) pages."""
    old_tables, old_lengths = [list(r) for r in tables], list(lengths)
    refs, tables, lengths = list(refs), [list(r) for r in tables], list(lengths)
    free_pages = [p for p, n in enumerate(refs) if n <= 0]
    seen, wanted, done, copies = set(), 0, [], []
    for a, c in zip(parents, children):
        good = 0 <= a < len(tables) and 0 <= c < len(tables) and c not in seen
        seen.add(c)
        good = good and old_lengths[c] == 0
        if good:
            n = min(max(old_lengths[a], 0), len(tables[a]) * ps)
            full, part = divmod(n, ps)
            good = not part or 0 <= old_tables[a][full] < len(refs)
        if not good:
            done.append(0)
            continue
        wanted += part > 0
        done.append(int(wanted <= len(free_pages)))
        if not done[-1]:
            continue
        row = old_tables[a][:full]
        for p in row:
            if 0 <= p < len(refs):
                refs[p] += 1
        if part:
            target = free_pages[wanted - 1]
            copies.append((old_tables[a][full], target))
            refs[target] = 1
            row = row + [target]
        tables[c], lengths[c] = row + [-1] * (len(tables[c]) - len(row)), n
    return refs, tables, lengths, done, copies


def compact(refs, tables):
    """(refs, tables, used, copies)."""
    refs, tables = list(refs), [list(r) for r in tables]
    used = sum(n > 0 for n in refs)
    holes = [p for p in range(used) if refs[p] <= 0]
    high = [p for p in range(used, len(refs)) if refs[p] > 0]
    to = dict(zip(high, holes))
    for a, z in to.items():
        refs[z], refs[a] = refs[a], 0
    return refs, [[to.get(p, p) for p in r] for r in tables], used, list(to.items())


def scores(logits, tokens, top):
    """(logprob, entropy, ids, top_logprobs) in binary64 by the definitions."""
    x = logits.detach().cpu().double()
    rows, n = x.shape
    out = [], [], [], []
    for r in range(rows):
        v = x[r]
        bad = bool(torch.isnan(v).any() or (v == math.inf).any())
        nothing = bool((v == -math.inf).all())
        key = torch.where(torch.isnan(v), math.inf, v)
        nan_first = torch.isnan(v).int()
        order = sorted(range(n), key=lambda i: (-nan_first[i].item(), -key[i].item(), i)) \
            if n <= 4096 else torch.sort(key, descending=True, stable=True).indices.tolist()
        ids = order[:top]
        # against the maximum: x - lse itself has no bits left under a mask of -3e38
        v = v - v.max()
        lse = torch.logsumexp(v, 0)
        token = int(tokens[r])
        if bad:
            lp = [math.nan] * top
            out[0].append(math.nan)
            out[1].append(math.nan)
        elif nothing:
            lp = [-math.inf] * top
            out[0].append(-math.inf if 0 <= token < n else math.nan)
            out[1].append(0.0)
        else:
            logp = v - lse
            p = torch.exp(logp)
            lp = logp[ids].tolist()
            out[0].append(logp[token].item() if 0 <= token < n else math.nan)
            out[1].append(-(p * torch.where(p > 0, logp, 0.0)).sum().item())
        out[2].append(ids)
        out[3].append(lp)
    return (torch.tensor(out[0], dtype=torch.float64), torch.tensor(out[1], dtype=torch.float64),
            torch.tensor(out[2], dtype=torch.int64).view(rows, top),
            torch.tensor(out[3], dtype=torch.float64).view(rows, top))
