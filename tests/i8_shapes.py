"""Token, channel and column counts for every way that the 8-bit integer calls
hand out their work: one shape for each (call, part of it, kernel, columns of a
tile, distribution) that the library's plan can choose.  Distributions: "full"
(whole tiles, every round full), "whole" (the last tiles whole on some workers),
"slots" (the last tiles in pieces, added through global memory), "runs" (equal
runs over the last tiles), "cluster n" (n pieces, added through shared memory);
"full+" where full rounds come before.  test_i8_abi.py checks the list against
mpq_i8_plan, test_gpu_i8_plans.py runs it.
"""


def distribution(work):
    """The distribution of one part of i8_plan's answer."""
    before = "full+" if work["full"] else ""
    if work["rem"] == 0:
        return "full"
    if work["cluster"]:
        return "cluster %d" % work["cuts"]
    return before + {0: "runs", 1: "whole"}.get(work["cuts"], "slots")


def classes(plan):
    """{part: (kernel, columns, distribution)} of i8_plan's answer."""
    return {part: (w["kernel"], w["columns"], distribution(w)) for part, w in plan.items()}


# (call, part): {(kernel, columns): {distribution: (M, N, K)}}
SHAPES = {
    ("gated", "product"): {
        ("stream", 16): {
            "cluster 2": (557, 157, 1665), "cluster 3": (616, 70, 1291), "cluster 4": (391, 65, 1337),
            "cluster 5": (329, 72, 1105), "cluster 6": (245, 66, 1103), "cluster 7": (1, 66, 782),
            "cluster 8": (1, 68, 953), "full": (591, 434, 68), "full+runs": (1, 28894, 3783),
            "full+slots": (1, 19403, 1923), "full+whole": (2379, 69, 70), "runs": (1, 9637, 3468),
            "slots": (2, 9238, 3642), "whole": (1, 66, 66),
        },
        ("stream", 32): {
            "cluster 2": (814, 131, 2742), "cluster 3": (1206, 65, 1930), "cluster 4": (856, 69, 1780),
            "cluster 5": (712, 77, 1619), "cluster 6": (523, 64, 2701), "cluster 8": (17, 996, 1196),
            "full": (2349, 137, 169), "full+runs": (20, 29792, 6691), "full+slots": (18, 19785, 3216),
            "full+whole": (2382, 132, 148), "runs": (19, 9550, 5393), "slots": (20, 9347, 9639),
            "whole": (2393, 71, 133),
        },
        ("stream", 64): {
            "cluster 2": (1413, 146, 3993), "cluster 3": (1281, 130, 2943), "cluster 4": (1653, 66, 3730),
            "cluster 5": (1444, 65, 3329), "cluster 6": (34, 1849, 2003), "cluster 8": (33, 1461, 2530),
            "full": (2336, 921, 187), "full+runs": (39, 28427, 7700), "full+slots": (33, 19882, 4482),
            "full+whole": (35, 25538, 66), "runs": (37, 9970, 6551), "slots": (36, 9418, 12202),
            "whole": (33, 12716, 75),
        },
        ("stream", 128): {
            "cluster 2": (72, 6592, 7220), "cluster 3": (66, 4460, 3450), "cluster 4": (68, 3488, 3067),
            "cluster 5": (2916, 65, 5869), "cluster 6": (65, 1958, 3083), "cluster 8": (65, 1300, 6170),
            "full": (126, 18855, 2383), "full+runs": (74, 29928, 9906), "full+slots": (77, 19071, 7310),
            "full+whole": (69, 26243, 142), "runs": (67, 9516, 9480), "whole": (65, 12777, 151),
        },
        ("tile", 256): {
            "full": (2467, 403, 133), "full+whole": (1865, 1677, 64),
        },
    },
    ("gated_backward", "gradient"): {
        ("dx", 32): {
            "full": (2342, 66, 131), "full+runs": (3, 1569, 28456), "full+slots": (2, 769, 20294),
            "full+whole": (258, 66, 3653), "runs": (270, 2603, 1107), "slots": (2, 840, 66), "whole": (1, 68, 67),
        },
        ("dx", 64): {
            "full": (2343, 66, 340), "full+runs": (41, 1975, 28589), "full+slots": (33, 1587, 19185),
            "full+whole": (2526, 70, 278), "runs": (2413, 2223, 65), "slots": (808, 2257, 70),
            "whole": (2390, 77, 66),
        },
        ("dx", 128): {
            "full": (459, 66, 9426), "full+runs": (297, 2777, 9627), "full+slots": (77, 1646, 19257),
            "full+whole": (76, 65, 19891), "runs": (2508, 2946, 272), "slots": (2649, 3607, 67),
            "whole": (2515, 146, 280),
        },
        ("dx", 256): {
            "full": (153, 171, 18761), "full+runs": (135, 2487, 28864), "full+slots": (143, 1609, 20997),
            "full+whole": (144, 75, 27854), "runs": (131, 2706, 9944), "slots": (2696, 11643, 67),
            "whole": (146, 64, 14179),
        },
    },
    ("gated_backward", "product"): {
        ("stream", 16): {
            "cluster 2": (520, 129, 1818), "cluster 3": (262, 129, 1390), "cluster 4": (436, 66, 1156),
            "cluster 5": (372, 66, 1043), "cluster 6": (227, 64, 1306), "cluster 7": (2, 64, 817),
            "cluster 8": (1, 65, 910), "full": (1175, 140, 87), "full+runs": (1, 28547, 3497),
            "full+slots": (1, 19368, 1949), "full+whole": (1235, 134, 69), "runs": (4, 9485, 3799),
            "slots": (1, 9333, 3699), "whole": (1, 68, 67),
        },
        ("stream", 32): {
            "cluster 2": (1589, 67, 2714), "cluster 3": (596, 143, 2056), "cluster 4": (414, 129, 1675),
            "cluster 5": (727, 66, 1541), "cluster 6": (531, 68, 2669), "cluster 8": (17, 926, 1271),
            "full": (2351, 165, 144), "full+runs": (19, 28453, 5437), "full+slots": (17, 19096, 3442),
            "full+whole": (2392, 129, 138), "runs": (17, 10154, 5173), "slots": (18, 9464, 8997),
            "whole": (1239, 129, 149),
        },
        ("stream", 64): {
            "cluster 2": (1452, 137, 4162), "cluster 3": (2619, 64, 2949), "cluster 4": (1696, 64, 3632),
            "cluster 5": (1412, 68, 3317), "cluster 6": (33, 1906, 1903), "cluster 8": (36, 1408, 2968),
            "full": (33, 18918, 129), "full+runs": (34, 29122, 6541), "full+slots": (36, 20266, 5368),
            "full+whole": (33, 28590, 70), "runs": (41, 9494, 6818), "slots": (35, 9331, 12671),
            "whole": (33, 12573, 84),
        },
        ("stream", 128): {
            "cluster 2": (69, 5875, 7139), "cluster 3": (70, 4402, 3596), "cluster 4": (66, 3826, 2852),
            "cluster 5": (1488, 144, 5736), "cluster 6": (67, 1918, 3773), "cluster 8": (66, 1508, 6225),
            "full": (90, 18872, 504), "full+runs": (68, 28653, 7673), "full+slots": (66, 19240, 6973),
            "full+whole": (69, 25689, 152), "runs": (66, 9840, 7644), "slots": (82, 9266, 29916),
            "whole": (66, 12966, 147),
        },
        ("tile", 256): {
            "full": (1910, 573, 131), "full+whole": (1481, 1994, 66),
        },
    },
    ("linear", "product"): {
        ("stream", 16): {
            "cluster 2": (1, 5636, 3520), "cluster 3": (568, 73, 3059), "cluster 4": (219, 130, 2655),
            "cluster 5": (328, 69, 2330), "cluster 6": (273, 66, 2414), "cluster 8": (2, 65, 1816),
            "full": (1184, 138, 142), "full+runs": (2, 29655, 10095), "full+slots": (1, 18954, 4673),
            "full+whole": (1291, 131, 65), "runs": (2, 9702, 8985), "slots": (2, 9458, 9038), "whole": (1, 65, 66),
        },
        ("stream", 32): {
            "cluster 2": (1046, 131, 5283), "cluster 3": (1029, 65, 4173), "cluster 4": (393, 129, 3799),
            "cluster 5": (737, 64, 3211), "cluster 6": (582, 66, 3930), "cluster 8": (387, 73, 4604),
            "full": (2363, 448, 84), "full+runs": (20, 28531, 11353), "full+slots": (17, 21240, 6856),
            "full+whole": (2371, 273, 65), "runs": (19, 9725, 10824), "slots": (20, 9272, 10934),
            "whole": (2369, 72, 272),
        },
        ("stream", 64): {
            "cluster 2": (1698, 136, 8233), "cluster 3": (1189, 146, 5440), "cluster 4": (815, 133, 5343),
            "cluster 5": (1425, 65, 5094), "cluster 6": (1026, 70, 8094), "cluster 8": (35, 1215, 3879),
            "full": (33, 18885, 87), "full+runs": (37, 29570, 15233), "full+slots": (35, 19211, 7685),
            "full+whole": (35, 19192, 65), "runs": (35, 10181, 12370), "slots": (35, 9449, 11262),
            "whole": (34, 13881, 68),
        },
        ("stream", 128): {
            "cluster 2": (2870, 131, 14026), "cluster 3": (2437, 131, 7785), "cluster 4": (1589, 137, 11186),
            "cluster 5": (1430, 132, 8311), "cluster 6": (71, 1897, 5558), "cluster 8": (67, 1691, 5143),
            "full": (93, 18839, 813), "full+runs": (259, 9491, 16343), "full+slots": (66, 19198, 9768),
            "full+whole": (66, 21441, 249), "runs": (76, 9691, 11867), "slots": (68, 9431, 19244),
            "whole": (67, 12665, 313),
        },
        ("tile", 256): {
            "full": (928, 9322, 75), "full+whole": (1727, 4271, 64),
        },
    },
    ("linear_backward", "gradient"): {
        ("dx", 32): {
            "full": (1158, 64, 324), "full+runs": (1, 3211, 28864), "full+slots": (1, 1680, 19365),
            "full+whole": (2645, 72, 68), "runs": (257, 5464, 1144), "slots": (1, 1764, 64), "whole": (1, 65, 68),
        },
        ("dx", 64): {
            "full": (2318, 135, 281), "full+runs": (35, 3921, 28759), "full+slots": (40, 2853, 19500),
            "full+whole": (2415, 65, 550), "runs": (2387, 5418, 68), "slots": (878, 4649, 67),
            "whole": (2442, 142, 73),
        },
        ("dx", 128): {
            "full": (94, 145, 18908), "full+runs": (66, 4801, 29447), "full+slots": (65, 2913, 22089),
            "full+whole": (68, 69, 27059), "runs": (2578, 5886, 273), "slots": (1577, 10559, 67),
            "whole": (65, 71, 13936),
        },
        ("dx", 256): {
            "full": (166, 284, 18792), "full+runs": (258, 6899, 14498), "full+slots": (130, 3371, 21642),
            "full+whole": (132, 130, 21929), "runs": (141, 5075, 10657), "slots": (132, 10205, 2101),
            "whole": (130, 132, 12899),
        },
    },
}


def cases():
    """(call, part, kernel, columns, distribution, M, N, K) of every shape."""
    return [(*call, *kernel, how, *shape) for call, kernels in SHAPES.items() for kernel, ways in kernels.items()
            for how, shape in ways.items()]
