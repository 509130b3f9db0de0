"""Calls of windowed attention and of attention over a shared prefix that reach kernels' forms of their own,
with the plan that each has on 256 compute units: test_attention_plans_host checks the plans,
test_gpu_attention_forms the results."""

# name: (queries, own keys, heads_q, heads_kv, head_dim, causal, (left, right, sinks) or prefix,
#        (kernel, waves, parts of a weight, shares of own keys, shares of the prefix))
FORMS = {
    # windows that limit one side only, or hold about all keys, keep the tile of 256 rows
    "window eight waves": ([254, 241], [254, 241], 96, 96, 128, False, (-1, 5, 0), ("rows", 8, 1, 1, 0)),
    "window eight waves right": ([254, 241], [254, 241], 96, 96, 96, False, (300, -1, 2), ("rows", 8, 1, 1, 0)),
    "window eight waves both": ([254, 241], [254, 241], 96, 96, 96, False, (190, 80, 3), ("rows", 8, 1, 1, 0)),
    # a cut-off prefix in attention_rows: own keys in one share, in two, in many
    "cut rows": ([4, 1, 6, 4, 0, 4, 9, 4, 4, 4], [40, 1, 6, 11, 3, 0, 9, 33, 4, 17], 8, 1, 128, True, 3000,
                 ("rows", 4, 1, 1, 12)),
    "cut rows 72": ([4, 1, 6, 4, 0, 4, 9, 4, 4, 4], [40, 1, 6, 11, 3, 0, 9, 33, 4, 17], 8, 1, 72, False, 3000,
                    ("rows", 4, 1, 1, 12)),
    "cut rows 64": ([2, 1, 3] * 6 + [1], [40, 1, 6] * 6 + [30], 16, 2, 64, False, 3000, ("rows", 4, 1, 2, 12)),
    "cut rows own shares": ([4, 1, 6, 4, 0, 4, 9, 4, 4, 4], [4000, 1, 600, 11, 3, 0, 2000, 33, 77, 1517], 8, 1, 128, True,
                            6000, ("rows", 4, 1, 32, 24)),
    "cut rows own shares 96": ([4, 1, 6, 4, 0, 4, 9, 4, 4, 4], [4000, 1, 600, 11, 3, 0, 2000, 33, 77, 1517], 8, 1, 96,
                               False, 6000, ("rows", 4, 1, 32, 24)),
    "cut rows own shares 64": ([4, 1, 6, 4, 0, 4, 9, 4, 4, 4], [4000, 1, 600, 11, 3, 0, 2000, 33, 77, 1517], 16, 2, 64,
                               True, 3000, ("rows", 4, 1, 32, 12)),
}

# New tokens, whose weights go in two parts.  Behind the plan: the most keys whose weights one wave adds up.
TOKENS = {
    "whole": ([1, 3, 1, 2], [300, 131, 31, 512], 8, 2, 128, True, (-1, -1, 0), ("keys", 4, 2, 1, 0), 512),
    "window": ([1, 2, 1], [390, 5, 700], 8, 2, 128, True, (200, 0, 9), ("keys", 4, 2, 1, 0), 212),
    "window 64": ([1, 3, 1, 2], [900, 300, 40, 77], 4, 4, 64, True, (250, 0, 4), ("keys", 4, 2, 1, 0), 257),
    "window shares": ([1, 3, 1], [5000, 700, 40], 8, 2, 128, True, (2000, 0, 4), ("keys", 4, 2, 23, 0), 256),
    "window shares two waves": ([1] * 12, [1500, 700, 40, 1, 1100, 256, 900, 5, 2000, 1021, 333, 800], 32, 8, 128, True,
                                (900, 0, 4), ("keys", 2, 2, 9, 0), 256),
    "window two waves": ([1, 3, 1], [100, 60, 77], 8, 2, 128, True, (90, 0, 4), ("keys", 2, 2, 1, 0), 97),
    "prefix": ([1, 2, 1, 3], [50, 300, 1, 3], 6, 3, 96, True, 150, ("keys", 4, 2, 1, 0), 450),
    "prefix 64": ([1, 2, 1, 3], [50, 300, 1, 3], 6, 3, 64, False, 150, ("keys", 4, 2, 1, 0), 450),
    "prefix cut": ([1, 2, 1, 1], [50, 700, 5, 3], 8, 2, 128, True, 3000, ("keys", 4, 2, 3, 12), 256),
    "prefix cut two waves": ([1, 2] * 7, [5, 70, 33, 2, 300, 7, 1] * 2, 24, 8, 96, True, 3000, ("keys", 2, 2, 4, 12), 256),
    "prefix cut 64": ([1] * 9, [7, 700, 5, 3, 1, 90, 33, 64, 300], 6, 3, 64, True, 3000, ("keys", 4, 2, 5, 12), 256),
}


def sizes(lq, lk, hq, hkv, d, causal, keys):
    """What a plan depends on: batch, total_q, total_k, heads, head_dim, causal, window and prefix."""
    window, prefix = (keys, 0) if isinstance(keys, tuple) else ((-1, -1, 0), keys)
    return (len(lq), sum(lq), sum(lk), hq, hkv, d, int(causal), *window, prefix)
