"""Sizes that give the workgroups of qlinear_w8a8's stream three tiles and more: (M, N, K, row stride, shape behind the
stream).  Units of 64 of K, an even number of them, move on by 2 (K 336) and by 0 of the ring's 4 slots; 1020 and 1450
tiles leave some workgroups one fewer; the strides of all but one are whole lines of 128 bytes in both types."""
STREAMS = [(7100, 7400, 336, 7424, 0), (7100, 7400, 464, 7424, 0), (13056, 5120, 336, 5120, 3), (12700, 7400, 400, 7424, 3),
           (9900, 7168, 480, 7168, 1), (17776, 5760, 336, 5760, 1), (7100, 7400, 336, 7403, 0)]
