"""Lists of matrices that, on 256 compute units, reach every tile of each product of the Muon update's larger matrices
(test_muon_plan.py shows it, test_gpu_muon.py runs them): (rows, cols) of each."""

LISTS = [
    [(131, 135)], [(129, 387)], [(2, 9001)],
    [(133, 917)] * 24, [(513, 3149)] * 2, [(401, 455)] * 24,
    [(129, 917)] * 48, [(391, 3836)] * 8, [(773, 959)] * 24,
    [(137, 133)], [(387, 138)], [(9001, 2)],
    [(455, 129)] * 48, [(2691, 535)] * 2, [(497, 401)] * 24,
    [(1991, 129)] * 24, [(3831, 385)] * 8, [(1047, 786)] * 24,
    # different sizes in one launch: padded to the same unit
    [(130 + 37 * k, 257 + 41 * k) for k in range(20)], [(300 + 61 * k, 131 + 53 * k) for k in range(20)],
]
