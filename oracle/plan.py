"""Plain definition of the page plan of a serving step, request by request (TEST INFRASTRUCTURE, see core.py; no
counterpart in the pages it cites).

A group is a dict: window, num_pages, table (list of lists), ring (list), pool [head, count], first (list or None),
lost (list or None), freed (list of lists of pages per request, or None). plan() changes the groups in place and
returns what the call writes besides.
"""
from __future__ import annotations

from typing import Sequence


def pages(tokens: int) -> int:
    return -(-tokens // 16)


def plan(ctx: Sequence[int], new: Sequence[int], rows: int, groups):
    """(ctx_len after, q_start, q_len, positions, [seq_len per group], [slots per group])."""
    n_req = len(ctx)
    for g in groups:
        g["want"], g["take"], g["back"] = 0, 0, []
        if g["lost"] is not None and g["freed"] is not None:
            g["lost"] = [x + 16 * len(f) for x, f in zip(g["lost"], g["freed"])]
    after, q_start, q_len, pos = list(ctx), [], [], [-1] * rows
    seq, slots = [[] for _ in groups], [[-1] * rows for _ in groups]
    at = 0
    for b in range(n_req):
        add = max(0, new[b])
        held = [ctx[b] - (g["lost"][b] if g["lost"] is not None else 0) for g in groups]
        ok = add > 0 and at + add <= rows
        for g, h in zip(groups, held):
            need = pages(h + add) - pages(h)
            g["want"] += need
            ok = ok and (need == 0 or g["want"] <= g["pool"][1])
        for i, (g, h) in enumerate(zip(groups, held)):
            if g["freed"] is not None:
                g["back"] += g["freed"][b]
            first = g["first"][b] if g["first"] is not None else 0
            to = pages(h) if new[b] < 0 else max(first, max(0, h - g["window"] + 1) // 16) if ok and g["window"] else first
            g["back"] += g["table"][b][first:to]
            if ok:
                for page in range(pages(h), pages(h + add)):
                    g["table"][b][page] = g["ring"][(g["pool"][0] + g["take"]) % g["num_pages"]]
                    g["take"] += 1
                for r in range(add):
                    slots[i][at + r] = 16 * g["table"][b][(h + r) // 16] + (h + r) % 16
            seq[i].append(h + add if ok else 0)
            if g["first"] is not None:
                g["first"][b] = 0 if new[b] < 0 else to
            if g["lost"] is not None and new[b] < 0:
                g["lost"][b] = 0
        if ok:
            pos[at:at + add] = range(ctx[b], ctx[b] + add)
        after[b] = 0 if new[b] < 0 else ctx[b] + (add if ok else 0)
        q_start.append(at)
        q_len.append(add if ok else 0)
        at += add
    for g in groups:
        for i, page in enumerate(g["back"]):
            g["ring"][(g["pool"][0] + g["pool"][1] + i) % g["num_pages"]] = page
        g["pool"] = [(g["pool"][0] + g["take"]) % g["num_pages"], g["pool"][1] - g["take"] + len(g["back"])]
    return after, q_start, q_len, pos, seq, slots
