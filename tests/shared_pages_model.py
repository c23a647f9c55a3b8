"""Pages with several holders, request by request in Python: what
fork_block_tables, release_shared_block_tables, compact_block_tables and
copy_cache_pages do, and a random pool to try them on."""
import numpy as np

import paged_attention_decode_split_gb300 as pa


def pages_of(n, bs):
    return -(-n // bs)


def clamp_pool(num_free, P):
    return min(max(num_free, 0), P), pa.PA_DEV_BAD_PAGE if not 0 <= num_free <= P else 0


def fork(lens, parent, table, free, num_free, shares, bs):
    """dict of the outputs, and the status."""
    B, width, P = len(lens), table.shape[1], len(free)
    pool, status = clamp_pool(num_free, P)
    out = dict(table=table.copy(), lens=np.maximum(lens, 0), shares=shares.copy(), src=np.full(B, -1, np.int32),
               dst=np.full(B, -1, np.int32), tokens=np.zeros(B, np.int32))
    wanted = taken = 0
    for b in range(B):
        a = parent[b]
        if a < 0:
            if lens[b] < 0 or lens[b] > width * bs:
                status |= pa.PA_DEV_BAD_SEQLEN
            continue
        ok = a < B and a != b and parent[a] < 0 and lens[b] == 0 and 0 <= lens[a] <= width * bs
        if not ok:
            status |= pa.PA_DEV_BAD_SEQLEN
            continue
        full, rest = divmod(int(lens[a]), bs)
        wanted += rest > 0
        if rest and wanted > pool:
            status |= pa.PA_DEV_NO_PAGES
            continue
        out["lens"][b] = lens[a]
        for k in range(full):
            page = out["table"][b, k] = table[a, k]
            if 0 <= page < P:
                out["shares"][page] += 1
            else:
                status |= pa.PA_DEV_BAD_PAGE
        if rest:
            page = free[pool - wanted]
            if not 0 <= page < P:
                status |= pa.PA_DEV_BAD_PAGE
            out["table"][b, full] = page
            out["src"][b], out["dst"][b], out["tokens"][b] = table[a, full], page, rest
            taken += 1
    return out | dict(num_free=pool - taken), status


def release(lens, finished, table, free, num_free, shares, bs):
    width, P = table.shape[1], len(free)
    pool, status = clamp_pool(num_free, P)
    out = dict(lens=np.where(finished != 0, 0, np.maximum(lens, 0)).astype(np.int32), shares=shares.copy(), free=free.copy())
    for b in range(len(lens)):
        if lens[b] < 0 or lens[b] > width * bs:
            status |= pa.PA_DEV_BAD_SEQLEN
            continue
        for k in range(pages_of(int(lens[b]), bs) if finished[b] else 0):
            if 0 <= table[b, k] < P:
                out["shares"][table[b, k]] -= 1
            else:
                status |= pa.PA_DEV_BAD_PAGE
    for page in np.nonzero(out["shares"] < 0)[0]:
        if out["shares"][page] < -1 or pool >= P:
            status |= pa.PA_DEV_BAD_PAGE
        out["shares"][page] = 0
        if pool < P:
            out["free"][pool] = page
            pool += 1
    return out | dict(num_free=pool), status


def compact(lens, table, free, num_free, shares, bs, most):
    width, P = table.shape[1], len(free)
    pool, status = clamp_pool(num_free, P)
    used = np.ones(P, bool)
    for page in free[:pool]:
        if 0 <= page < P:
            used[page] = False
        else:
            status |= pa.PA_DEV_BAD_PAGE
    n = int(used.sum())
    where, shares = np.arange(P, dtype=np.int32), shares.copy()
    src, dst = np.full(most, -1, np.int32), np.full(most, -1, np.int32)
    for k in range(most):
        high = np.nonzero(used)[0]
        low = np.nonzero(~used)[0]
        low = low[~np.isin(low, src)]  # (a page that has just been left is not filled again)
        if not len(high) or high[-1] < n or not len(low) or low[0] >= n:
            break
        src[k], dst[k] = high[-1], low[0]
        used[src[k]], used[dst[k]] = False, True
        where[src[k]] = dst[k]
        shares[dst[k]], shares[src[k]] = shares[src[k]], 0
    out = dict(src=src, dst=dst, map=where, shares=shares, table=table.copy())
    out["free"] = np.full(P, -1, np.int32)
    left = np.nonzero(~used)[0][::-1]
    out["free"][:len(left)] = left
    for b in range(len(lens)):
        if lens[b] < 0 or lens[b] > width * bs:
            status |= pa.PA_DEV_BAD_SEQLEN
            continue
        for k in range(pages_of(int(lens[b]), bs)):
            if 0 <= table[b, k] < P:
                out["table"][b, k] = where[table[b, k]]
            else:
                status |= pa.PA_DEV_BAD_PAGE
    return out | dict(num_free=len(left), extent=int(used.nonzero()[0].max()) + 1 if used.any() else 0), status


def pool(rng, B, width, bs, spare, share=0.5):
    """Random requests over a pool of scattered pages, some holding a stretch of full pages of an earlier one:
    dict of lens, table, free, num_free, shares."""
    lens = rng.integers(0, width * bs + 1, B).astype(np.int32)
    lens[rng.random(B) < 0.2] = 0
    P = int(sum(pages_of(int(n), bs) for n in lens)) + spare
    order, at = rng.permutation(P).astype(np.int32), 0
    table = rng.integers(-5, P + 5, (B, width)).astype(np.int32)  # what is not in use may be anything
    holders = np.zeros(P, np.int64)
    for b in range(B):
        have = pages_of(int(lens[b]), bs)
        common = 0
        if b and rng.random() < share:
            a = int(rng.integers(0, b))
            common = int(rng.integers(0, min(lens[a], lens[b]) // bs + 1))
            table[b, :common] = table[a, :common]
        table[b, common:have] = order[at:at + have - common]
        at += have - common
        np.add.at(holders, table[b, :have], 1)
    free = np.full(P, -1, np.int32)
    free[:P - at] = order[at:]
    return dict(lens=lens, table=table, free=free, num_free=P - at, shares=np.maximum(holders - 1, 0).astype(np.int32))
