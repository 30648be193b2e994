"""The KV split of the attention over lists, seen through the workspace that it asks
for: partial results of each split behind the lists.  No GPU is needed."""
from test_serving_refusals import lib  # noqa: F401


def splits(lib, B, n, Hq, Hkv, dh, top, max_pages, P, mt):  # noqa: F811
    """S of a call whose groups have mt * 128 query rows (1: none is split)."""
    up = lambda x: (x + 255) // 256 * 256
    G, rows = Hq // Hkv, n * (Hq // Hkv)
    groups = B * Hkv * -(-rows // (128 * mt))
    nodes = min(n, (128 * mt + G - 2) // G + 1)
    stride = min(max_pages, nodes * top)
    lists = up(groups * 4) + up(groups * stride * 4) + up(groups * nodes * -(-stride // 32) * 4)
    got = lib.eagle_tree_attn_kv8_pages_workspace_size(1, B, n, Hq, Hkv, dh, top, max_pages, P) - lists
    part = groups * min(-(-rows // 8) * 8, 128 * mt) * (dh + 2) * 4
    assert got >= 0 and got % part == 0
    return max(1, got // part)


def test_one_sequence_whose_nodes_may_share_nothing(lib):  # noqa: F811
    """Groups that leave most SMs idle: split for the longest list there can be."""
    assert splits(lib, 1, 49, 64, 8, 128, 4, 132, 16, 2) >= 4      # 16 groups of up to 132 pages of 16
    assert splits(lib, 1, 256, 8, 8, 64, 8, 1024, 16, 2) >= 4      # 8 groups of up to 1024
    assert splits(lib, 1, 61, 32, 32, 128, 4, 256, 16, 1) >= 4     # 32 groups of up to 244


def test_groups_that_fill_the_machine_are_not_split(lib):  # noqa: F811
    assert splits(lib, 16, 49, 64, 8, 128, 16, 128, 64, 2) == 1
    assert splits(lib, 64, 61, 64, 8, 64, 8, 64, 128, 2) == 1


def test_a_table_no_longer_than_a_tile_is_not_split(lib):  # noqa: F811
    assert splits(lib, 1, 49, 64, 8, 128, 4, 4, 16, 2) == 1
