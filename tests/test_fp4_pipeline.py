"""The order of accesses to what the roles of the attention-weights kernel share, without a GPU.

The roles' operations are taken from the source in the order in which they stand, laid out
over a few tiles, and joined by what each barrier phase orders: a wait comes after all
arrivals of its phase.  A word that one role writes and another reads has to be ordered by
that alone.
"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_norm_rope_gb300", "csrc")
TILES = 14


def _body(text, name):
    """The function's body: from its name to the first closing brace in column 0."""
    start = text.index(f"void {name}(")
    return text[start:text.index("\n}\n", start)]


def _in_order(body, operations):
    """Names of the operations by where each (last) stands in the text."""
    at = {name: [m.start() for m in re.finditer(pattern, body)] for name, pattern in operations.items()}
    assert all(at.values()), at
    return sorted(at, key=lambda name: at[name][-1])


def _reaches(edges, start, end):
    todo, seen = [start], set()
    while todo:
        node = todo.pop()
        if node == end:
            return True
        if node not in seen:
            seen.add(node)
            todo += edges.get(node, [])
    return False


def test_weights_kernel_orders_the_words_of_valid_keys():
    with open(os.path.join(CSRC, "fp4_weights.cu")) as f:
        text = f.read()
    slots = int(re.search(r"kOkTiles = (\d+);", text).group(1))
    convert = _in_order(_body(text, "convert_role"), {
        "write": r"s\.key_ok\[[^;]*\] = ", "wait staged_free": r"mbar_wait\(&s\.staged_free",
        "arrive staged": r"mbar_arrive\(&s\.staged\["})
    multiply = _in_order(_body(text, "multiply_role"), {
        "wait scores_free": r"mbar_wait\(&s\.scores_free", "wait staged": r"mbar_wait\(&s\.staged\[",
        "arrive staged_free": r"mma_commit\(&s\.staged_free", "arrive scores": r"mma_commit\(&s\.scores\["})
    add = _in_order(_body(text, "sum_role"), {
        "wait scores": r"mbar_wait\(&s\.scores\[", "arrive scores_free": r"mbar_arrive\(&s\.scores_free",
        "read": r"s\.key_ok\["})
    # the tile whose phase a wait of tile t is for (two places of scores, one of keys)
    behind = {"staged_free": 1, "scores_free": 2, "staged": 0, "scores": 0}
    edges = {}
    for role, operations in (("convert", convert), ("multiply", multiply), ("add", add)):
        line = [(role, t, name) for t in range(TILES) for name in operations]
        for a, b in zip(line, line[1:]):
            edges.setdefault(a, []).append(b)
        for t in range(TILES):
            for name in operations:
                if name.startswith("wait "):
                    barrier = name[5:]
                    source = {"staged_free": "multiply", "scores": "multiply", "staged": "convert",
                              "scores_free": "add"}[barrier]
                    if t >= behind[barrier]:
                        edges.setdefault((source, t - behind[barrier], "arrive " + barrier), []).append((role, t, name))
    for t in range(TILES):
        assert _reaches(edges, ("convert", t, "write"), ("add", t, "read")), t
        if t >= slots:
            # the word's next use comes after the last one's reads
            assert _reaches(edges, ("add", t - slots, "read"), ("convert", t, "write")), t
