"""Sizes that the GPU tests of the log probabilities run, and that a CPU test
(tests/test_beside_sizes.py) holds against the rules that choose the kernels."""

# rows, vocabulary: a workgroup of 256, 512 and 1,024 threads a row, of one segment, of some and with
# groups of several, and rows in parts
LOGPROB_ROWS = [(513, 20011), (513, 70001), (520, 157184), (260, 30011), (260, 140001), (129, 40007), (129, 270001), (5, 5003), (7, 9001),
                (3, 157184), (64, 40001), (2, 1000003)]
