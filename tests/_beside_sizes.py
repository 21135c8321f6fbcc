"""Sizes that the GPU tests of the log probabilities run, and that a CPU test
(tests/test_beside_sizes.py) holds against the rules that choose the kernels."""

# rows, vocabulary: a workgroup of 256, 512 and 1,024 threads a row, of one segment, of some and with
# groups of several, and rows in parts
LOGPROB_ROWS = [(513, 20011), (513, 70001), (520, 157184), (260, 30011), (260, 140001), (129, 40007), (129, 270001), (5, 5003), (7, 9001),
                (3, 157184), (64, 40001), (2, 1000003)]
# a wave a row: of a segment and of two to six
LOGPROB_SHORT_ROWS = [(3, 1), (70, 40), (5, 300), (40, 1000), (33, 1024), (9, 1025), (600, 2048), (520, 4095), (1025, 5000), (1030, 6001)]


def lora_tokens(rank):
    """The fewest tokens of that rank that always go to the matrix cores."""
    return 16384 // (-(-rank // 32) * 32) + 8


# (tokens, rank, in_features, out_features) on the matrix cores: ranks, depths and channels at every way they
# are read, with and without adapters dealt to several workgroups
LORA_RANKS = [(lora_tokens(r), r, 72, 67) for r in (1, 2, 3, 5, 7, 8, 9, 12, 13, 15, 16, 17, 20, 24, 25, 31, 32, 33, 40, 47, 63, 64, 65, 71, 95,
                                                     96, 97, 104, 113, 127, 128)]
LORA_DEPTHS = [(lora_tokens(r), r, K, 80) for r in (13, 16, 40) for K in (1, 2, 3, 7, 8, 9, 31, 33, 63, 64, 65, 127, 511, 513, 769, 1000, 2561)]
LORA_CHANNELS = [(lora_tokens(r), r, 48, N) for r in (6, 11, 16, 64) for N in (1, 2, 3, 4, 5, 8, 15, 47, 63, 65, 255, 257, 1001)]
LORA_LARGE = [(4200, 16, 72, 40), (4101, 13, 65, 300), (16400, 3, 40, 257), (2100, 64, 130, 4100), (1030, 128, 96, 1300)]
