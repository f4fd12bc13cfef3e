// A stand-in for the HIP runtime on the host: libqmv.so and libqmx.so, loaded
// after this library with global symbols, launch into it.  Nothing runs; each
// launch and function attribute is kept as a line of text.
#include <cstdio>
#include <cstring>
#include <map>
#include <string>

#include <hip/hip_runtime_api.h>

static std::map<const void *, std::string> &names()
{
    static std::map<const void *, std::string> m;
    return m;
}
static std::string &lines()
{
    static std::string s;
    return s;
}
static int device = 0;
static char taken[256];

extern "C" {

const char *rec_lines() { return lines().c_str(); }
void rec_clear() { lines().clear(); }

void **__hipRegisterFatBinary(const void *)
{
    static void *module = taken;
    return &module;
}
void __hipRegisterFunction(void **, const void *host, char *, const char *name, unsigned, void *, void *, void *,
                           void *, int *)
{
    names()[host] = name;
}
void __hipRegisterVar(void **, void *, char *, char *, int, size_t, int, int) {}
void __hipUnregisterFatBinary(void **) {}
hipError_t __hipPopCallConfiguration(dim3 *, dim3 *, size_t *, hipStream_t *) { return hipSuccess; }

hipError_t hipGetDevice(int *d)
{
    *d = device;
    return hipSuccess;
}
hipError_t hipSetDevice(int d)
{
    device = d;
    return hipSuccess;
}
hipError_t hipStreamGetDevice(hipStream_t, hipDevice_t *d)
{
    *d = device;
    return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int *v, hipDeviceAttribute_t, int)
{
    *v = 256;                                     // compute units of an MI355X
    return hipSuccess;
}
hipError_t hipOccupancyMaxActiveBlocksPerMultiprocessor(int *n, const void *, int, size_t)
{
    *n = 2;
    return hipSuccess;
}
hipError_t hipMemPoolCreate(hipMemPool_t *p, const hipMemPoolProps *)
{
    *p = (hipMemPool_t)taken;
    return hipSuccess;
}
hipError_t hipMemPoolSetAttribute(hipMemPool_t, hipMemPoolAttr, void *) { return hipSuccess; }
hipError_t hipMallocFromPoolAsync(void **p, size_t, hipMemPool_t, hipStream_t)
{
    *p = taken;
    return hipSuccess;
}
hipError_t hipFreeAsync(void *, hipStream_t) { return hipSuccess; }
hipError_t hipGetSymbolAddress(void **p, const void *)
{
    *p = taken;
    return hipSuccess;
}

static void line(const char *what, const void *fn, const char *rest)
{
    lines() += std::string(what) + " " + std::to_string(device) + " " + names()[fn] + " " + rest + "\n";
}
hipError_t hipFuncSetAttribute(const void *fn, hipFuncAttribute attr, int value)
{
    char b[64];
    std::snprintf(b, sizeof b, "%d", attr == hipFuncAttributeMaxDynamicSharedMemorySize ? value : -1);
    line("attr", fn, b);
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void *fn, dim3 g, dim3 t, void **, size_t lds, hipStream_t)
{
    char b[128];
    std::snprintf(b, sizeof b, "%u %u %u %u %zu", g.x, g.y, g.z, t.x * t.y * t.z, lds);
    line("launch", fn, b);
    return hipSuccess;
}

}  // extern "C"
