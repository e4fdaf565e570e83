/* What a host-only compilation of HIP sources asks of the runtime, so that their host functions run
 * without it: registering kernels does nothing, and launching one ends the program. */
#include <stdlib.h>

void* __hipRegisterFatBinary(const void* data) { return (void*)data; }
void __hipUnregisterFatBinary(void* modules) { (void)modules; }
void __hipRegisterFunction(void) {}
int __hipPushCallConfiguration(void) { abort(); }
int __hipPopCallConfiguration(void) { abort(); }
int hipLaunchKernel(void) { abort(); }
int hipGetLastError(void) { return 0; }
