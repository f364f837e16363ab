"""Oracle: pages that sequences share, and accepted drafts moved together.

Test infrastructure only (see ``oracle/__init__``).  Plain Python over block tables
(lists of lists), lengths and counts, in place; page bytes through ``layout``.
Every function returns the status bits that its inputs call for.

Parity: pinned (tests/test_oracle_pages.py) by hand cases and by counts that have
to add up after random calls.
"""

import numpy as np

from . import layout

BAD_PAGE, BAD_SEQ, NO_PAGES = 0x2, 0x4, 0x20
PAGE = layout.PAGE_TOKENS


def _free(refs):
    return [p for p, n in enumerate(refs) if n == 0]


def extend(refs, table, lens, new, n_tokens):
    """Grows sequence b by new[b] tokens, or none where one would shrink; (slots [n_tokens], status)."""
    status, slots, free, dry, back = 0, [], _free(refs), False, min(new, default=0) < 0
    for b, n in enumerate(new):
        row = table[b]
        if n < 0 or lens[b] < 0 or lens[b] + n > len(row) * PAGE:
            status |= BAD_SEQ
            slots += [-1] * max(n, 0)
            continue
        if n and lens[b] % PAGE and row[lens[b] // PAGE] < 0:
            status |= BAD_PAGE
            slots += [-1] * n
            continue
        if back:
            continue
        blocks = {p // PAGE for p in range(lens[b], lens[b] + n)} - ({lens[b] // PAGE} if lens[b] % PAGE else set())
        short = [i for i in sorted(blocks) if row[i] < 0]
        dry = dry or len(short) > len(free)
        if short and dry:
            status |= NO_PAGES
            slots += [-1] * n
            continue
        for i in short:
            row[i] = free.pop(0)
            refs[row[i]] = 1
        slots += [row[p // PAGE] * PAGE + p % PAGE for p in range(lens[b], lens[b] + n)]
        lens[b] += n
    return [-1] * n_tokens if back else slots + [-1] * (n_tokens - len(slots)), status


def fork(refs, table, lens, src, dst):
    """(copies [(from, to, tokens)], status)."""
    status, copies, free = 0, [], _free(refs)
    old_lens, old_table = list(lens), [list(r) for r in table]
    taken = set()
    for a, b in zip(src, dst):
        if not (0 <= a < len(table) and 0 <= b < len(table)) or old_lens[b] or max(old_table[b]) >= 0 or b in taken:
            status |= BAD_SEQ
            continue
        taken.add(b)
        n, row = old_lens[a], old_table[a]
        rest = n % PAGE
        if rest and not 0 <= row[n // PAGE] < len(refs):
            status |= BAD_PAGE
            continue
        if rest and not free:
            status |= NO_PAGES
            continue
        new = row[: n // PAGE]
        for p in new:
            if 0 <= p < len(refs):
                refs[p] += 1
            else:
                status |= BAD_PAGE
        if rest:
            page = free.pop(0)
            refs[page] = 1
            copies.append((row[n // PAGE], page, rest))
            new = new + [page]
        table[b][:] = new + [-1] * (len(row) - len(new))
        lens[b] = n
    return copies, status


def release(refs, table, lens, rows):
    status = 0
    for b in rows:
        if not 0 <= b < len(table):
            status |= BAD_SEQ
            continue
        for i, p in enumerate(table[b]):
            if p < 0:
                continue
            table[b][i] = -1
            if p < len(refs) and refs[p] > 0:
                refs[p] -= 1
            else:
                status |= BAD_PAGE
        lens[b] = 0
    return status


def token_bytes(kv, idx, slot):
    """What the pools hold at a slot: codes, scales and index key of one token."""
    return layout.read_kv_slot(kv, slot // PAGE, slot % PAGE), layout.read_index_slot(idx, slot // PAGE, slot % PAGE)


def put_token(kv, idx, slot, token):
    layout.write_kv_slot(kv, slot // PAGE, slot % PAGE, *token[0])
    layout.write_index_slot(idx, slot // PAGE, slot % PAGE, token[1])


def copy(kv, idx, copies):
    """The first tokens of pages, one layer."""
    for a, b, tokens in copies:
        held = [token_bytes(kv, idx, a * PAGE + t) for t in range(tokens)]
        for t, x in enumerate(held):
            put_token(kv, idx, b * PAGE + t, x)


def commit(kv, idx, table, lens, drafts, accepted):
    """(new lengths, status) of one layer's pools, in place."""
    status, new_lens = 0, list(lens)
    n_pages = np.asarray(kv).shape[0]
    for b, n in enumerate(drafts):
        if n < 0 or n > 64 or n > lens[b] or lens[b] > len(table[b]) * PAGE:
            status |= BAD_SEQ
            continue
        ctx = lens[b] - n
        kept = [j for j in range(n) if accepted[b] >> j & 1]
        new_lens[b] = ctx + len(kept)
        held = []
        for k, j in enumerate(kept):
            if k == j:
                continue
            a, z = table[b][(ctx + j) // PAGE], table[b][(ctx + k) // PAGE]
            if not (0 <= a < n_pages and 0 <= z < n_pages):
                status |= BAD_PAGE
                continue
            held.append((z * PAGE + (ctx + k) % PAGE, token_bytes(kv, idx, a * PAGE + (ctx + j) % PAGE)))
        for slot, x in held:
            put_token(kv, idx, slot, x)
    return new_lens, status
