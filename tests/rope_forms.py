"""Calls of the norm and rotation of queries and keys whose waves take two, three and four steps of heads:
test_attention_plans_host checks that they do, test_gpu_qk_norm_rope_steps the results."""

# lengths of the packed sequences, heads of queries and keys, head_dim, steps of a wave
CASES = [
    ([700], 24, 24, 128, 2),
    ([1, 0, 1311, 64, 700, 0, 3], 8, 8, 128, 2),
    ([2049, 77], 7, 3, 72, 2),
    ([63, 2100, 1], 13, 2, 64, 2),
    ([1100], 24, 24, 128, 3),
    ([77, 699, 1, 401, 154, 50], 21, 5, 128, 3),
    ([0, 900, 0, 1200, 5], 11, 9, 72, 3),
    ([2100], 5, 3, 256, 3),
    ([1050, 1051], 130, 150, 8, 3),
    ([77, 899, 1, 701, 154, 250], 16, 16, 72, 4),
    ([1, 1100, 2, 300], 32, 8, 128, 4),
    ([700, 0, 0, 1433], 13, 5, 128, 4),
    ([2051], 30, 6, 40, 4),
    ([1] * 2100, 16, 3, 128, 4),
]


def launch_of(rows, hq, hk, d, steps):
    """Workgroups of four waves that a launch has whose waves take `steps` steps of 64 / lanes heads."""
    lanes = 1
    while 8 * lanes < d:
        lanes *= 2
    heads = steps * (64 // lanes)
    return -(-rows * (-(-hq // heads) + -(-hk // heads)) // 4)
