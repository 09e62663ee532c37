"""A shape for every compiled variant of the 4-bit products: (x loads, column blocks, waves, blocks per step) ->
(M, N, K, gated). Rows fewer than the variant's, column blocks that no workgroup's number of them divides, an odd
last block, and K of three steps and a cut one in each wave's share or so."""
PLAIN = {
    (0, 1, 16, 1): (1, 67), (0, 2, 8, 1): (1, 8225), (0, 2, 4, 2): (1, 8225),
    (1, 1, 16, 1): (3, 67), (1, 4, 4, 1): (3, 8241),
    (4, 1, 8, 1): (9, 67), (4, 2, 8, 1): (16, 8225), (4, 4, 8, 1): (9, 16401),
    (8, 1, 8, 1): (20, 67), (8, 2, 8, 1): (32, 8225), (8, 4, 8, 1): (20, 12305),
    (16, 1, 8, 1): (40, 67), (16, 2, 4, 1): (64, 8225), (16, 4, 4, 1): (64, 12305),
}
GATED = {
    (0, 2, 16, 1): (1, 37), (0, 2, 8, 1): (1, 4129), (0, 2, 4, 2): (1, 4129), (1, 2, 16, 1): (4, 37), (1, 4, 4, 1): (3, 4129),
    (4, 2, 8, 1): (11, 37), (4, 4, 8, 1): (16, 8209), (8, 2, 8, 1): (25, 37), (8, 4, 8, 1): (32, 8209),
    (16, 2, 4, 1): (50, 37), (16, 4, 4, 1): (64, 8209),
}


def shapes():
    """(variant, M, N, K, gated): N is F where gated."""
    for table, gated in ((PLAIN, False), (GATED, True)):
        for v, (M, N) in table.items():
            # the single row on pairs and 8 waves serves K from 32 blocks on
            yield v, M, N, 4128 if v == (0, 2, 8, 1) else v[2] * v[3] * 384 + 96, gated
