"""Sizes that the GPU tests of the log probabilities run, and that a CPU test
(tests/test_beside_sizes.py) holds against the rules that choose the kernels."""

# rows, vocabulary: a workgroup of 256, 512 and 1,024 threads a row, of one segment, of some and with
# groups of several, and rows in parts
LOGPROB_ROWS = [(513, 20011), (513, 70001), (520, 157184), (260, 30011), (260, 140001), (129, 40007), (129, 270001), (5, 5003), (7, 9001),
                (3, 157184), (64, 40001), (2, 1000003)]
# a wave a row: of a segment and of two to six
LOGPROB_SHORT_ROWS = [(3, 1), (70, 40), (5, 300), (40, 1000), (33, 1024), (9, 1025), (600, 2048), (520, 4095), (1025, 5000), (1030, 6001)]
